// Packing into and reading back of the block-scaled formats (block.cuh has the arithmetic).
//
// Packing is one pass over x.  A CTA takes a tile of 128 rows, so that the scales it makes are
// whole 512-byte scale tiles that it writes in one run:
//   along the rows: each lane holds 32 bytes of a row; the lanes of a block (one or two for bf16,
//     two or four for fp32) share its amax by shuffles, so values go from registers to codes with
//     no second read.  (16 bytes of bf16 a lane took 59 us where this takes 50, 8190 x 14336; 64 bytes
//     of fp32 89 us against 81, 4096 x 28672.)
//   along the columns (the transposed output): the tile is kept in shared memory; a thread then
//     walks 32 rows of its column(s), lanes on neighbouring columns (no bank conflicts), and the
//     codes go out through a second small stage, 64 bytes of a transposed row at a time.
// Both outputs cost one read of x.  Rows alone are bound by memory: 8190 x 14336 bf16 takes 47 us to
// MXFP4 (94% of the copy rate), 50 to NVFP4 (89%), 53 to MXFP8 (99%); 4096 x 28672 fp32 77 us to MXFP4
// (101%), 80 to NVFP4 (99%), 84 to MXFP8 (103%).  Both ways are bound by instructions, about 8 an element
// for each way: 70 us (76%), NVFP4 84 (64%), fp32 115 (76%) and 132 (67%).  Reading back is bound by its
// writes: 49 us (89%), NVFP4 51 (86%), MXFP8 57 (92%).
#include "block.cuh"
#include "cast.cuh"

namespace te {
namespace {

constexpr int kThreads = 256;
constexpr int kTileRows = 128;

// 32 rows of a tile held in shared memory, of the kCols neighbouring columns that a thread walks.
template <typename T>
struct Strip;
template <>
struct Strip<__nv_bfloat16> {
  static constexpr int kCols = 2;
  uint32_t w[32];  // both columns of a row
  __device__ __forceinline__ void load(const uint8_t* p, int pitch) {
#pragma unroll
    for (int r = 0; r < 32; ++r) w[r] = *reinterpret_cast<const uint32_t*>(p + r * pitch);
  }
  __device__ __forceinline__ float at(int k, int r) const { return k ? bf16_hi(w[r]) : bf16_lo(w[r]); }
  // bits of the largest magnitudes of rows [r0, r0 + N), one a column
  template <int N>
  __device__ __forceinline__ void amax_bits(int r0, uint32_t (&m)[2]) const {
    // 32 rows: both columns at once in 16 bits (73 us against 77, MXFP4 8190 x 14336 both ways), 16
    // rows: in fp32, three values an instruction (80 us against 93 for NVFP4)
    if constexpr (N == 32) {
      uint32_t t = 0;
#pragma unroll
      for (int r = 0; r < N; ++r) t = __vmaxu2(t, w[r0 + r] & 0x7fff7fffu);
      m[0] = t << 16;
      m[1] = t & 0xffff0000u;
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < N; r += 2) t = max_abs3(t, at(k, r0 + r), at(k, r0 + r + 1));
        m[k] = __float_as_uint(t);
      }
    }
  }
};
template <>
struct Strip<float> {
  static constexpr int kCols = 1;
  float v[32];
  __device__ __forceinline__ void load(const uint8_t* p, int pitch) {
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] = *reinterpret_cast<const float*>(p + r * pitch);
  }
  __device__ __forceinline__ float at(int, int r) const { return v[r]; }
  template <int N>
  __device__ __forceinline__ void amax_bits(int r0, uint32_t (&m)[1]) const {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < N; r += 2) t = max_abs3(t, v[r0 + r], v[r0 + r + 1]);
    m[0] = __float_as_uint(t);
  }
};

constexpr int kColTile = 128;           // columns of a tile that is also packed along its columns
constexpr int kStagePitch = 64 + 16;    // bytes of a transposed row's codes in shared memory

template <typename T>
__host__ __device__ constexpr int tile_pitch() { return kColTile * int(sizeof(T)) + 16; }
template <typename T>
__host__ __device__ constexpr size_t col_smem() { return size_t(kTileRows) * tile_pitch<T>() + kColTile * kStagePitch; }

// Threads of a CTA: for tiles packed along their columns a strip of 32 rows each.
template <typename T, bool COL>
__host__ __device__ constexpr int quant_threads() { return COL && sizeof(T) == 4 ? 512 : kThreads; }

// TC: columns of a tile (256 when only the rows are packed, for whole 128-byte runs of codes).
// SUB: rows of the tile that a CTA takes, 128, or 32 (rows only) so that few rows still occupy many
// SMs; such a CTA writes the 4 bytes of each 16 of a scale tile that are its rows'.
template <typename T, int FMT, int TC, bool COL, int SUB>
__global__ void __launch_bounds__(quant_threads<T, COL>()) block_quantize_kernel(BlockQuantArgs a) {
  constexpr int THREADS = quant_threads<T, COL>();
  static_assert(SUB == kTileRows || (SUB == 32 && !COL), "rows of a CTA");
  constexpr int kBlk = block_len(FMT);
  constexpr int kPer = sizeof(T) == 2 ? 2 : 1;   // vectors of 8 that a lane holds: 32 bytes of x
  constexpr int kLanes = TC / (8 * kPer);        // lanes on one row
  constexpr int kRowsPass = THREADS / kLanes;   // rows a CTA takes at a time
  constexpr int kPasses = SUB / kRowsPass;
  constexpr int kBatch = kPasses < 4 ? kPasses : 4;  // passes whose loads are in flight together
  constexpr int kScaleBytes = kTileRows * (TC / kBlk);
  __shared__ __align__(16) uint8_t rs[kScaleBytes];
  __shared__ __align__(16) uint8_t cs[COL ? kScaleBytes : 16];
  __shared__ float sums[COL ? 4 : 1][COL ? kColTile : 1];
  __shared__ float factors[FMT == TE_NVFP4 ? kNvFactors : 1];
  extern __shared__ __align__(16) uint8_t dyn[];
  // the kernel after this one may launch its setup now (it waits for this grid's completion)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float s = 1.0f;
  if constexpr (FMT == TE_NVFP4) {
    s = a.amax_in ? nv_scale_from_amax(*a.amax_in) : *a.scale;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      if (a.scale_out) *a.scale_out = s;
      if (a.scale_inv_out) *a.scale_inv_out = __fdiv_rn(1.0f, s);
    }
    nv_factors(factors, s, int(threadIdx.x), THREADS);
    __syncthreads();
  }
  const int64_t tiles_c = (a.N + TC - 1) / TC;
  // after a pass for the amax the last tiles first: those of them that it left in L2 are read there
  // (8190 x 14336 bf16 with that pass 91 -> 82 us, both ways 128 -> 123)
  const int64_t tile_id = FMT == TE_NVFP4 && a.amax_in ? int64_t(gridDim.x) - 1 - blockIdx.x : int64_t(blockIdx.x);
  const int64_t st = tile_id / tiles_c, ct = tile_id % tiles_c;
  const int64_t rt = st / (kTileRows / SUB);
  const int sub = int(st % (kTileRows / SUB));
  const int64_t r0 = st * SUB, c0 = ct * TC;
  const int cl = int(threadIdx.x) % kLanes * (8 * kPer);  // this lane's column within the tile
  const bool col_ok = c0 + cl < a.N;             // whole vectors; whole blocks where rows are packed
  const int rl = int(threadIdx.x) / kLanes;
  const T* x = static_cast<const T*>(a.x) + r0 * a.N + c0 + cl;
  uint8_t* tile = dyn;
  const int64_t pitch = a.N / codes_per_byte(FMT);
  uint8_t* codes = static_cast<uint8_t*>(a.codes) + r0 * pitch + (c0 + cl) / codes_per_byte(FMT);
  uint32_t amax = 0;
  const int rows = col_ok ? int(min(int64_t(SUB), a.M - r0)) : 0;  // of this lane's column
#pragma unroll 1
  for (int p0 = 0; p0 < kPasses; p0 += kBatch) {
    Eight<T> e[kBatch][kPer];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = (p0 + j) * kRowsPass + rl;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (r < rows) e[j][k].load(x + int64_t(r) * a.N + 8 * k);
        else e[j][k].zero();
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = (p0 + j) * kRowsPass + rl;
      if constexpr (COL) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) e[j][k].to_smem(tile + r * tile_pitch<T>() + (cl + 8 * k) * int(sizeof(T)));
      }
      if (COL && !a.codes && !a.amax_out) continue;
      uint32_t m = e[j][0].amax_bits();
      if constexpr (kPer == 2) m = max(m, e[j][kPer - 1].amax_bits());
#pragma unroll
      for (int o = 1; o * 8 * kPer < kBlk; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (a.amax_out) amax = max(amax, m <= kInfBits ? m : 0u);  // blocks with a NaN left out
      if (!COL || a.codes) {
        const bool in = r < rows;
        const BlockScale b = block_scale<FMT>(m, s, factors);
        if (in) {
          uint2 c[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            float v[8];
            e[j][k].get(v);
            c[k] = codes8<FMT>(v, b);
          }
          uint8_t* out = codes + r * pitch;
          if constexpr (FMT == TE_MXFP8) {
            if constexpr (kPer == 2) *reinterpret_cast<uint4*>(out) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
            else *reinterpret_cast<uint2*>(out) = c[0];
          } else {
            if constexpr (kPer == 2) *reinterpret_cast<uint2*>(out) = make_uint2(c[0].x, c[1].x);
            else *reinterpret_cast<uint32_t*>(out) = c[0].x;
          }
        }
        if (cl % kBlk == 0) rs[scale_offset(r, cl / kBlk)] = in ? uint8_t(b.byte) : uint8_t(0);
      }
    }
  }
  __syncthreads();
  // the tile's scale tiles, those of them that the row of tiles has
  if (!COL || a.codes) {
    const int64_t groups = scale_groups(FMT, a.N);
    const int64_t g0 = c0 / kBlk / 4;
    const int n = int(min(int64_t(kScaleBytes), (groups - g0) * 512));
    uint8_t* dst = static_cast<uint8_t*>(a.scales) + (rt * groups + g0) * 512;
    if constexpr (SUB == kTileRows) {
      for (int i = int(threadIdx.x) * 16; i < n; i += THREADS * 16)
        *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(rs + i);
    } else {  // the rows r % 32 lie in words 0, 4, 8, ... of rs
      for (int i = int(threadIdx.x) * 16; i < n; i += THREADS * 16)
        *reinterpret_cast<uint32_t*>(dst + i + sub * 4) = *reinterpret_cast<const uint32_t*>(rs + i);
    }
  }
  if constexpr (COL) {
    constexpr int kC = Strip<T>::kCols;
    uint8_t* stage = dyn + kTileRows * tile_pitch<T>();
    // (column(s), 32 rows) for every thread
    static_assert(kColTile / kC * 4 == THREADS, "one strip a thread");
    const int c = int(threadIdx.x) % (kColTile / kC) * kC, rb = int(threadIdx.x) / (kColTile / kC);
    Strip<T> v;
    v.load(tile + rb * 32 * tile_pitch<T>() + c * int(sizeof(T)), tile_pitch<T>());
    const bool rows_in = r0 + rb * 32 < a.M;
    if (a.partials) {
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += v.at(k, r);
        sums[rb][c + k] = t;
      }
    }
#pragma unroll
    for (int h = 0; h < 32 / kBlk; ++h) {
      uint32_t m[kC];
      v.template amax_bits<kBlk>(h * kBlk, m);
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        const BlockScale b = block_scale<FMT>(m[k], s, factors);
        cs[scale_offset(c + k, rb * (32 / kBlk) + h)] = rows_in && c0 + c + k < a.N ? uint8_t(b.byte) : uint8_t(0);
        uint32_t q[kBlk / 8];
#pragma unroll
        for (int g = 0; g < kBlk / 8; ++g) {
          float w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = v.at(k, h * kBlk + g * 8 + i);
          q[g] = codes8<FMT>(w, b).x;
        }
        uint8_t* d = stage + (c + k) * kStagePitch + rb * 16 + h * 8;
        if constexpr (kBlk == 32) *reinterpret_cast<uint4*>(d) = make_uint4(q[0], q[1], q[2], q[3]);
        else *reinterpret_cast<uint2*>(d) = make_uint2(q[0], q[1]);
      }
    }
    __syncthreads();
    const int64_t mp = (a.M + 31) / 32 * 32;
    const int64_t pitch_t = a.pitch_t ? a.pitch_t : mp / 2;
    const int64_t groups = scale_groups(FMT, mp);
    const int64_t g0 = r0 / kBlk / 4;
    const int n = int(min(int64_t(kScaleBytes), (groups - g0) * 512));
    uint8_t* dst = static_cast<uint8_t*>(a.scales_t) + (ct * groups + g0) * 512;
    for (int i = int(threadIdx.x) * 16; i < n; i += THREADS * 16)
      *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(cs + i);
    // 16 bytes of codes (32 rows) for each of 4 lanes on a transposed row
    for (int u = int(threadIdx.x); u < kColTile * 4; u += THREADS) {
      const int c = u / 4, rb = u % 4;
      if (c0 + c < a.N && r0 + rb * 32 < mp)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.codes_t) + (c0 + c) * pitch_t + r0 / 2 + rb * 16) =
            *reinterpret_cast<const uint4*>(stage + c * kStagePitch + rb * 16);
    }
    if (a.partials)
      for (int c = int(threadIdx.x); c < kColTile; c += THREADS)
        if (c0 + c < a.N)
          a.partials[rt * a.N + c0 + c] = ((sums[0][c] + sums[1][c]) + sums[2][c]) + sums[3][c];
  }
  if (a.amax_out) block_amax_commit(__uint_as_float(amax), a.amax_out);
}

template <typename T, int FMT>
te_status launch_quant_t(const BlockQuantArgs& a, cudaStream_t s) {
  const bool col = a.codes_t != nullptr;
  const int64_t tc = col ? kColTile : 256;
  const int64_t tiles = ceil_div(a.M, kTileRows) * ceil_div(a.N, tc);
  if (tiles > 0x1fffffff) return TE_ERR_UNSUPPORTED;
  if (!col) {
    // 32-row CTAs throughout for fp32 and for MXFP8, whole tiles for bf16 to 4 bits once there are enough
    // of them for every SM.  32-row CTAs against whole tiles, us:
    //   tiles          64         160        320        448        512        1024       4096
    //   bf16 MXFP4   2.0  3.1   3.0  4.1   4.7  5.3   5.9  5.5   6.5  6.4  12.2 10.3  53.8 50.1
    //   bf16 NVFP4   2.6  3.5   3.6  4.4   5.4  5.4   6.7  5.6   7.5  6.5  14.3 10.7  58.3 51.4
    //   bf16 MXFP8   2.1  3.4   3.0  4.3   4.3  5.4   5.3  5.4   5.9  6.7  12.7 13.9  57.7 58.4
    //   fp32 MXFP4   2.7  5.1   3.9  6.1   5.5  7.7   6.8  7.8   7.8  9.5  23.6 25.1  84.9 86.1
    //   fp32 NVFP4   3.1  5.7   4.5  6.8   6.4  8.3   8.2  8.3   9.1 10.0  24.5 27.1  86.4 92.1
    //   fp32 MXFP8   2.8  5.0   4.0  6.1   5.6  7.7   7.0  7.8   8.2  9.7  25.6 26.9  93.7 94.6
    // (MXFP4 crosses at 288, back at 320, and for good after 480; NVFP4 at 240.)
    if constexpr (sizeof(T) == 2 && FMT != TE_MXFP8) {
      if (2 * tiles >= (FMT == TE_NVFP4 ? 3 : 6) * num_sms()) {
        block_quantize_kernel<T, FMT, 256, false, kTileRows><<<unsigned(tiles), kThreads, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
      }
    }
    block_quantize_kernel<T, FMT, 256, false, 32><<<unsigned(tiles * 4), kThreads, 0, s>>>(a);
  } else if constexpr (FMT == TE_MXFP8) {
    return TE_ERR_UNSUPPORTED;  // checkpoints are read along their rows only
  } else {
    static PerDevice<bool> attr_set;
    bool ok = false;
    if (!attr_set.get(&ok, [](bool* v) {
          *v = cudaFuncSetAttribute(block_quantize_kernel<T, FMT, kColTile, true, kTileRows>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(col_smem<T>())) == cudaSuccess;
          return *v;
        }))
      return TE_ERR_CUDA;
    block_quantize_kernel<T, FMT, kColTile, true, kTileRows>
        <<<unsigned(tiles), quant_threads<T, true>(), col_smem<T>(), s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

// ------------------------------------------------------------------ the tensor's amax -----

// max |x| of `vectors` vectors of 8, NaN ignored, by one integer atomic a CTA.  Four vectors a thread
// are in flight; all of a wave's threads stride together.
constexpr int kAmaxBatch = 4;
constexpr int kAmaxCtas = 8;  // CTAs of an SM

template <typename T>
__global__ void __launch_bounds__(kThreads) amax_kernel(const void* x, int64_t vectors, float* amax_out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  float m[kAmaxBatch] = {};
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < vectors; i += kAmaxBatch * stride) {
    Eight<T> e[kAmaxBatch];
#pragma unroll
    for (int j = 0; j < kAmaxBatch; ++j) {
      if (i + j * stride < vectors) e[j].load(static_cast<const T*>(x) + (i + j * stride) * 8);
      else e[j].zero();
    }
#pragma unroll
    for (int j = 0; j < kAmaxBatch; ++j) m[j] = fmaxf(m[j], e[j].amax());
  }
  block_amax_commit(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), amax_out);
}

// ------------------------------------------------------------------ reading back ----------

// A tile of 128 rows x 256 columns a CTA: its scales first, in one run, then 8 codes a lane.
template <int FMT, typename OutT>
__global__ void __launch_bounds__(kThreads) block_dequantize_kernel(BlockDequantArgs a) {
  constexpr int TC = 256;
  constexpr int kBlk = block_len(FMT);
  constexpr int kScaleBytes = kTileRows * (TC / kBlk);
  constexpr int kPasses = kTileRows / (kThreads / 32);
  constexpr int kBatch = 8;  // a lane's loads are 4 or 8 bytes: many rows in flight
  __shared__ __align__(16) uint8_t rs[kScaleBytes];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t tiles_c = (a.N + TC - 1) / TC;
  const int64_t rt = blockIdx.x / tiles_c, ct = blockIdx.x % tiles_c;
  const int64_t r0 = rt * kTileRows, c0 = ct * TC;
  const int64_t groups = scale_groups(FMT, a.N);
  const int64_t g0 = c0 / kBlk / 4;
  const int n = int(min(int64_t(kScaleBytes), (groups - g0) * 512));
  const uint8_t* src = static_cast<const uint8_t*>(a.scales) + (rt * groups + g0) * 512;
  for (int i = int(threadIdx.x) * 16; i < n; i += kThreads * 16)
    *reinterpret_cast<uint4*>(rs + i) = __ldg(reinterpret_cast<const uint4*>(src + i));
  const float inv = a.scale_inv ? *a.scale_inv : 1.0f;
  const int cl = int(threadIdx.x) % 32 * 8;
  const int rl = int(threadIdx.x) / 32;
  const int64_t pitch = a.N / codes_per_byte(FMT);
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes) + r0 * pitch + (c0 + cl) / codes_per_byte(FMT);
  OutT* out = static_cast<OutT*>(a.out) + r0 * a.N + c0 + cl;
  __syncthreads();
  if (c0 + cl >= a.N) return;
  CastState none;
#pragma unroll 1
  for (int p0 = 0; p0 < kPasses; p0 += kBatch) {
    uint2 w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = (p0 + j) * (kThreads / 32) + rl;
      w[j] = make_uint2(0u, 0u);
      if (r0 + r < a.M) {
        if constexpr (FMT == TE_MXFP8) w[j] = __ldg(reinterpret_cast<const uint2*>(codes + r * pitch));
        else w[j].x = __ldg(reinterpret_cast<const uint32_t*>(codes + r * pitch));
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = (p0 + j) * (kThreads / 32) + rl;
      if (r0 + r >= a.M) break;
      const uint32_t sb = rs[scale_offset(r, cl / kBlk)];
      const f32x2 f = f2s(FMT == TE_NVFP4 ? unpack_e4m3x2(uint16_t(sb)).x : e8m0_value(sb));
      f32x2 v[4];
      if constexpr (FMT == TE_MXFP8) {
        v[0] = unpack_e4m3x2(uint16_t(w[j].x));
        v[1] = unpack_e4m3x2(uint16_t(w[j].x >> 16));
        v[2] = unpack_e4m3x2(uint16_t(w[j].y));
        v[3] = unpack_e4m3x2(uint16_t(w[j].y >> 16));
      } else {
        unpack_e2m1x8(w[j].x, v);
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x2 t = mul2(v[i], f);  // exact
        if constexpr (FMT == TE_NVFP4) t = mul2(t, f2s(inv));
        y[2 * i] = f2lo(t);
        y[2 * i + 1] = f2hi(t);
      }
      store_out<sizeof(OutT) == 4 ? OUT_F32 : OUT_BF16, 8>(out, int64_t(r) * a.N, y, none);
    }
  }
}

template <int FMT>
te_status launch_dequant_t(const BlockDequantArgs& a, unsigned tiles, cudaStream_t s) {
  if (a.out_dtype == TE_F32) block_dequantize_kernel<FMT, float><<<tiles, kThreads, 0, s>>>(a);
  else block_dequantize_kernel<FMT, __nv_bfloat16><<<tiles, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

}  // namespace

te_status launch_block_quantize(const BlockQuantArgs& a, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_QUANTIZE, s);
  const bool f32 = a.x_dtype == TE_F32;
  switch (a.fmt) {
    case TE_MXFP4:
      return f32 ? launch_quant_t<float, TE_MXFP4>(a, s) : launch_quant_t<__nv_bfloat16, TE_MXFP4>(a, s);
    case TE_NVFP4:
      return f32 ? launch_quant_t<float, TE_NVFP4>(a, s) : launch_quant_t<__nv_bfloat16, TE_NVFP4>(a, s);
    default:
      return f32 ? launch_quant_t<float, TE_MXFP8>(a, s) : launch_quant_t<__nv_bfloat16, TE_MXFP8>(a, s);
  }
}

te_status launch_amax(const void* x, int x_dtype, int64_t n, float* amax_out, cudaStream_t s) {
  if (cudaMemsetAsync(amax_out, 0, sizeof(float), s) != cudaSuccess) return TE_ERR_CUDA;
  ProfileScope prof(TE_KERNEL_QUANTIZE, s);
  const int64_t vectors = n / 8, wave = int64_t(num_sms()) * kAmaxCtas;
  const int64_t need = ceil_div(vectors, kThreads * kAmaxBatch);
  const unsigned grid = unsigned(need < wave ? need : wave);
  if (x_dtype == TE_BF16) amax_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(x, vectors, amax_out);
  else amax_kernel<float><<<grid, kThreads, 0, s>>>(x, vectors, amax_out);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

te_status launch_block_dequantize(const BlockDequantArgs& a, cudaStream_t s) {
  const int64_t tiles = ceil_div(a.M, kTileRows) * ceil_div(a.N, 256);
  if (tiles == 0) return TE_OK;
  if (tiles > 0x7fffffff) return TE_ERR_UNSUPPORTED;
  ProfileScope prof(TE_KERNEL_QUANTIZE, s);
  switch (a.fmt) {
    case TE_MXFP4: return launch_dequant_t<TE_MXFP4>(a, unsigned(tiles), s);
    case TE_NVFP4: return launch_dequant_t<TE_NVFP4>(a, unsigned(tiles), s);
    default: return launch_dequant_t<TE_MXFP8>(a, unsigned(tiles), s);
  }
}

}  // namespace te

// The dense layer that ends in the residual stream, for a few tokens (up to 32 rows):
//   out = a residual + gate act(alpha x W + b)
// Reading W [K, N] once bounds it, so W goes straight from memory into the registers that the tensor
// cores read: a lane loads 16 bytes of a row of W at a time (8 bf16 or 16 E4M3 columns; of E4M3 beyond 8
// tokens 8 bytes, for the registers), four neighbouring rows k .. k + 3 for each step of 16, and pairs
// two rows' values of a column by byte permutes (E4M3 values become f16, exactly: with mma.sync on E4M3
// itself, which needs the bytes of four rows together, 17 tokens through [14336, 4096] took 25 us for 21).
// W is the first operand of mma.sync m16n8k16, so that a product takes two columns of each of the 8 lane
// groups as its 16 rows and 8 tokens as its columns; which row of W is which k of the product does not
// matter as long as x is read in the same order.  mma.sync rather than tcgen05: the arithmetic is far
// from any bound, and no weight passes through shared memory.
//
// A CTA of 8 warps takes the 64 (E4M3 up to 8 tokens: 128) columns of one lane's width, its warps different
// ranges of K, and a cluster of CTAs the ranges of one block of columns, where the columns alone leave SMs
// idle.  The partial sums meet in shared memory and over the cluster in a fixed order.  One token through
// [14336, 4096]: 24 us a call, 4.9 TB/s; about 4 of them are launch, first bytes and the sums' way.
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "sync.cuh"
#include "umma.cuh"

namespace te {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

struct FewArgs {
  const void* x;
  const void* w;
  const float* x_scale_inv;
  const float* w_scale_inv;
  const void* bias;
  const void* gate;
  const void* residual;
  void* out;
  void* z;
  float residual_scale;
  int out_dtype, act;
  int M, N, K, gate_rows;
};

// Two CTAs to an SM throughout, with as many loads in flight as their registers leave room for (one CTA of
// twice the registers: 36 to 39 us for 27 to 29, 32 tokens in E4M3 through [14336 to 16384, 4096], and 40
// for 36, 32 in bf16 through [8192, 8192]).  Staged in shared memory by asynchronous copies instead, which
// leave room for twice the bytes, one token through [14336, 4096] took 35 us for 24.
template <bool FP8, int XT>
struct Form {
  static constexpr int kWords = FP8 && XT > 1 ? 2 : 4;  // of 4 bytes, of a row of W to a lane
  static constexpr int kLane = kWords * (FP8 ? 4 : 2);  // columns of them
  static constexpr int kCols = 8 * kLane;               // of a CTA
  static constexpr int kPitch = kCols + 4;              // floats from row to row of a partial sum
  static constexpr int kAhead = XT == 1 ? 4 : XT == 4 ? 2 : FP8 && XT == 2 ? 4 : !FP8 && XT == 3 ? 2 : 3;  // steps in flight
  static constexpr int kCtas = 2;                       // of an SM
};

template <bool FP8, int XT>
constexpr size_t smem_bytes() { return size_t(kWarps / 2) * 8 * XT * Form<FP8, XT>::kPitch * sizeof(float); }

template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (FP8)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ int cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return int(n);
}

// (The kernel starts while the one in front may still write its inputs: ordinary loads throughout, behind
// the wait.)
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {  // of the low 16 bits
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(v)));
  return r;
}

// x's values of four neighbouring k: two operand registers.
template <bool FP8>
struct XFrag {
  uint2 w;  // bf16: four values; E4M3: four in w.x
  __device__ __forceinline__ void load(const void* x, int64_t at, bool in) {
    w = make_uint2(0u, 0u);
    if (!in) return;
    if constexpr (FP8) w.x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(x) + at);
    else w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + at);
  }
  __device__ __forceinline__ void get(uint32_t& lo, uint32_t& hi) const {
    if constexpr (FP8) {
      lo = e4m3x2_f16x2(w.x);
      hi = e4m3x2_f16x2(w.x >> 16);
    } else {
      lo = w.x;
      hi = w.y;
    }
  }
};

// XT: groups of 8 tokens.
template <bool FP8, int XT>
__global__ void __launch_bounds__(kThreads, Form<FP8, XT>::kCtas) dense_few_kernel(const FewArgs a) {
  using F = Form<FP8, XT>;
  constexpr int kAhead = F::kAhead, LW = F::kWords;
  constexpr int NP = F::kLane / 2;  // products of a step for each group of tokens: a pair of the lane's columns
  constexpr int ROWS = 8 * XT;
  extern __shared__ __align__(16) float part[];  // [4][ROWS][kPitch]
  // launched as a programmatic dependent: nothing is read before the kernel in front has finished
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int ranks = cluster_ctas(), rank = int(cluster_rank());
  const int col0 = int(blockIdx.x) / ranks * F::kCols;
  const int col = col0 + g * F::kLane;  // the lane's columns (N is a multiple of 16: all of them or none)
  const bool in = col < a.N;
  const int steps = a.K / 16, share = ranks * kWarps, id = rank * kWarps + warp;
  const int s0 = int(int64_t(steps) * id / share), s1 = int(int64_t(steps) * (id + 1) / share);
  constexpr int es = FP8 ? 1 : 2;
  const size_t row_bytes = size_t(a.N) * es;
  const uint8_t* wp = static_cast<const uint8_t*>(a.w) + (size_t(s0) * 16 + 4 * t) * row_bytes + size_t(col) * es;
  uint32_t w[kAhead][4][LW];
  XFrag<FP8> x[kAhead][XT];
  auto load = [&](int s, int b) {
    const uint8_t* p = wp + size_t(s - s0) * 16 * row_bytes;
    const bool here = s < s1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      using V = std::conditional_t<LW == 4, uint4, uint2>;
      V v{};
      if (here && in) v = *reinterpret_cast<const V*>(p + i * row_bytes);
      memcpy(w[b][i], &v, sizeof(V));
    }
#pragma unroll
    for (int r = 0; r < XT; ++r) {
      const int row = g + 8 * r;
      x[b][r].load(a.x, int64_t(row) * a.K + s * 16 + 4 * t, here && row < a.M);
    }
  };
  float acc[XT][NP][4];
#pragma unroll
  for (int m = 0; m < XT; ++m)
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
#pragma unroll
  for (int b = 0; b < kAhead; ++b) load(s0 + b, b);
  for (int s = s0; s < s1; s += kAhead) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      uint32_t xb[XT][2];
#pragma unroll
      for (int m = 0; m < XT; ++m) x[b][m].get(xb[m][0], xb[m][1]);
      const auto &r0 = w[b][0], &r1 = w[b][1], &r2 = w[b][2], &r3 = w[b][3];
#pragma unroll
      for (int q = 0; q < LW; ++q) {
        if constexpr (FP8) {
          const uint32_t lo[2] = {__byte_perm(r0[q], r1[q], 0x5140), __byte_perm(r0[q], r1[q], 0x7362)};
          const uint32_t hi[2] = {__byte_perm(r2[q], r3[q], 0x5140), __byte_perm(r2[q], r3[q], 0x7362)};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t wa[4] = {e4m3x2_f16x2(lo[j]), e4m3x2_f16x2(lo[j] >> 16), e4m3x2_f16x2(hi[j]),
                                    e4m3x2_f16x2(hi[j] >> 16)};
#pragma unroll
            for (int m = 0; m < XT; ++m) mma<FP8>(acc[m][2 * q + j], wa, xb[m]);
          }
        } else {
          const uint32_t wa[4] = {__byte_perm(r0[q], r1[q], 0x5410), __byte_perm(r0[q], r1[q], 0x7632),
                                  __byte_perm(r2[q], r3[q], 0x5410), __byte_perm(r2[q], r3[q], 0x7632)};
#pragma unroll
          for (int m = 0; m < XT; ++m) mma<FP8>(acc[m][q], wa, xb[m]);
        }
      }
      load(s + b + kAhead, b);
    }
  }
  // The lane's sums: of tokens 2 t and 2 t + 1 (of each group), product j gives its columns 2 j (c = 0, 1)
  // and 2 j + 1 (c = 2, 3).  The upper warps' first, then each lower warp's with its upper one's added.
  auto slab = [&](int s, int row, int c) { return part + (size_t(s) * ROWS + row) * F::kPitch + c; };
  auto rows_of = [&](auto&& f) {
#pragma unroll
    for (int m = 0; m < XT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < NP; j += 2) {
          float* p = slab(warp & 3, 8 * m + 2 * t + e, g * F::kLane + 2 * j);
          f(reinterpret_cast<float4*>(p), acc[m][j][e], acc[m][j][2 + e], acc[m][j + 1][e], acc[m][j + 1][2 + e]);
        }
  };
  if (warp >= 4) rows_of([](float4* p, float u, float v, float y, float z) { *p = make_float4(u, v, y, z); });
  __syncthreads();
  if (warp < 4)
    rows_of([](float4* p, float u, float v, float y, float z) {
      const float4 o = *p;
      *p = make_float4(u + o.x, v + o.y, y + o.z, z + o.w);
    });
  if (ranks > 1) cluster_sync();
  else __syncthreads();
  float alpha = 1.0f;
  if (a.x_scale_inv) alpha *= *a.x_scale_inv;
  if (a.w_scale_inv) alpha *= *a.w_scale_inv;
  // four neighbouring columns of a row to a thread of the cluster
  for (int i = rank * kThreads + int(threadIdx.x); i < a.M * (F::kCols / 4); i += ranks * kThreads) {
    const int row = i / (F::kCols / 4), c = i % (F::kCols / 4) * 4;
    if (col0 + c >= a.N) continue;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = 0; r < ranks; ++r) {
#pragma unroll
      for (int s = 0; s < kWarps / 2; ++s) {
        float4 p;
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w)
                     : "r"(map_to_rank(smem_u32(slab(s, row, c)), uint32_t(r)))
                     : "memory");
        v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
      }
    }
    const int64_t at = int64_t(row) * a.N + col0 + c;
    auto bf4 = [](const void* base, int64_t j) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + j);
      return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
    };
    const float4 b = a.bias ? bf4(a.bias, col0 + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(v[k], alpha, bb[k]);
    if (a.z)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.z) + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    const f32x2 v01 = act2(a.act, f2(v[0], v[1])), v23 = act2(a.act, f2(v[2], v[3]));
    float o[4] = {v01.x, v01.y, v23.x, v23.y};
    if (a.gate) {
      const float4 q = bf4(a.gate, int64_t(row / a.gate_rows) * a.N + col0 + c);
      o[0] *= q.x; o[1] *= q.y; o[2] *= q.z; o[3] *= q.w;
    }
    if (a.out_dtype == TE_BF16) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.residual) + at);
      const float r[4] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = fmaf(a.residual_scale, r[k], o[k]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    } else {
      const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + at);
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
          make_float4(fmaf(a.residual_scale, r.x, o[0]), fmaf(a.residual_scale, r.y, o[1]),
                      fmaf(a.residual_scale, r.z, o[2]), fmaf(a.residual_scale, r.w, o[3]));
    }
  }
  __syncwarp();
  if (ranks > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

template <bool FP8, int XT>
te_status launch(const FewArgs& f, cudaStream_t s) {
  constexpr size_t smem = smem_bytes<FP8, XT>();
  static PerDevice<bool> attr_done;
  bool ok = false;
  if (!attr_done.get(&ok, [](bool* v) {
        *v = cudaFuncSetAttribute(dense_few_kernel<FP8, XT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) ==
             cudaSuccess;
        return *v;
      }))
    return TE_ERR_CUDA;
  // CTAs to a block of columns: as many as keep every SM at the CTAs it holds at once, while each warp has
  // a round of loads to itself
  const int blocks = int(ceil_div(f.N, int64_t(Form<FP8, XT>::kCols)));
  const int64_t room = int64_t(num_sms()) * Form<FP8, XT>::kCtas;
  int ranks = 1;
  while (ranks < kMaxCluster && int64_t(blocks) * ranks * 2 <= room && f.K / 16 >= ranks * 2 * kWarps) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, dense_few_kernel<FP8, XT>, f) == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

}  // namespace

// Up to 8 rows always.  Each further group of 8 repeats the products of every weight, while the tiles of
// launch_gemm (256 columns wide, 128 rows high) cost the same for 1 row and for 128 and gain with their
// number: from about 6 / 5 tiles and groups an SM on they are faster.  Measured (us, here / tiles), bf16,
// K = 4096: N = 28672 (112 tiles) 48 / 62 at 8 rows, 55 / 44 at 16; N = 14336 (56) 28 / 38 at 16, 36 / 38
// at 32; K = 14336, N = 4096 (16) 24 / 55 at one row, 33 / 55 at 32.  E4M3 likewise: 27 / 34, 37 / 35;
// 20 / 25, 28 / 25; 17 / 40, 27 / 40.
bool dense_few_serves(int64_t M, int64_t N) {
  const int64_t groups = ceil_div(M, int64_t(8));
  return groups <= 1 || (groups <= 4 && ceil_div(N, int64_t(256)) * groups * 5 < int64_t(num_sms()) * 6);
}

te_status launch_dense_few(const GemmArgs& g, cudaStream_t s) {
  if (g.M == 0) return TE_OK;
  if (g.M > 32 || g.epilogue != EPI_RESIDUAL || g.N > (1 << 30) || g.K > (1 << 30)) return TE_ERR_UNSUPPORTED;
  ProfileScope prof(TE_KERNEL_GEMM_ACT, s);
  FewArgs f;
  f.x = g.A;
  f.w = g.B;
  f.x_scale_inv = g.a_scale_inv;
  f.w_scale_inv = g.b_scale_inv;
  f.bias = g.bias;
  f.gate = g.gate;
  f.residual = g.residual;
  f.out = g.D;
  f.z = g.saved_h;
  f.residual_scale = g.residual_scale;
  f.out_dtype = g.cast.out_dtype;
  f.act = g.act;
  f.M = int(g.M);
  f.N = int(g.N);
  f.K = int(g.K);
  f.gate_rows = int(g.gate_rows);
  const int groups = int(ceil_div(g.M, int64_t(8)));
  if (g.ab_dtype == TE_E4M3)
    return groups == 1 ? launch<true, 1>(f, s) : groups == 2 ? launch<true, 2>(f, s)
           : groups == 3 ? launch<true, 3>(f, s) : launch<true, 4>(f, s);
  return groups == 1 ? launch<false, 1>(f, s) : groups == 2 ? launch<false, 2>(f, s)
         : groups == 3 ? launch<false, 3>(f, s) : launch<false, 4>(f, s);
}

}  // namespace te

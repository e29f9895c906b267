// The dense layer that ends in the residual stream, for an output of few tiles (decoding, short prompts,
// narrow layers):
//   out = a residual + gate act(alpha x W + b)
// and its gradient dx = alpha dz W^T (the same kernel with W's rows for columns and nothing to join).
// Reading W [K, N] once bounds it.  The tiles of the batch product (128 tokens x 256 columns, an SM pair to
// two) leave most SMs idle here.  So W takes the 128-row side of tcgen05.mma and the tokens (rounded up to
// 32, 64 or 128) its columns, and a cluster splits K: each CTA multiplies its range of K into tensor
// memory and leaves its partial tile in shared memory, and the CTAs add the partial tiles in rank order
// through distributed shared memory, each finishing its share of the tile.  No sum depends on timing.
//
//   warp 0     TMA producer: a ring of W tiles (as stored, [K, N]: the MMA reads them transposed) and x tiles
//   warp 1     owns the tensor memory; one thread issues the MMAs
//   warps 2-9  bring the accumulator to shared memory, a TMEM lane quadrant to two warps
// and all of them finish the tile.
// Every wait on an mbarrier is bounded; on expiry a thread records TE_ERR_TIMEOUT, all roles leave their
// loops, and the CTA goes on to the cluster's barriers, behind the first of which no CTA of the cluster writes
// results.
//
// W [14336, 4096] (us; in brackets the time of its bytes at the measured copy rate): bf16 at 1, 32 and 128
// tokens 21, 23 and 28 (17.3, 17.5, 18.2); E4M3 13, 15 and 20 (8.7, 8.8, 9.2).  About 4 us of each are the
// launch, the first bytes and the meeting of the cluster (a [512, 512] layer takes 3.6); from 64 tokens on
// the x tiles add to the bytes on their way to shared memory and the end sums 8 partial tiles.  A first form,
// on mma.sync with W in registers, took 23 at one token and 33 at 32 (bf16), 16 and 27 (E4M3).  Starting
// each block of columns at another place of K, so that they do not all ask for the same x, is slower (13 ->
// 14 us in E4M3); four places at a time to a thread of the end gains nothing; ten warps for six are 1 to 3
// us faster from 128 tokens on, whose end is bound by instructions.
#include <cuda.h>

#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "sync.cuh"
#include "umma.cuh"

namespace te {

namespace {

constexpr int kCols = 128;       // columns of W to a CTA: the MMA's rows
constexpr int kRowBytes = 128;   // bytes of K (x) or of columns (W) to a row of a tile
constexpr int kThreads = 320;
constexpr int kWTile = kCols * kRowBytes;  // 16 KB: 64 (bf16) or 128 (E4M3) rows of W
constexpr int kPitch = kCols + 4;          // floats from token to token of a partial tile
constexpr int kMaxCluster = 8;

template <bool FP8, int NT>
struct Form {
  static constexpr int kK = kRowBytes / (FP8 ? 1 : 2);  // K of a stage
  static constexpr int kXTile = NT * kRowBytes;
  static constexpr int kStage = kWTile + kXTile;
  static constexpr int kStages = 100 * 1024 / kStage;   // two CTAs to an SM
  static constexpr size_t kRing = size_t(kStages) * kStage;
  static constexpr size_t kSums = size_t(NT) * kPitch * sizeof(float);
  static constexpr size_t kSmem = (kRing > kSums ? kRing : kSums) + 1024;  // (the ring starts on 1 KB)
};

// What ends the layer, for four neighbouring columns of a row to a thread.  (Ordinary loads throughout: the
// kernel in front may have written any of it.)
struct End {
  const float* x_scale_inv;
  const float* w_scale_inv;
  const void* bias;
  const void* gate;
  const void* residual;
  void* out;
  void* z;
  float residual_scale;
  int out_dtype, act;
  int N, gate_rows, one_gate;

  struct In {
    uint2 bias, gate;
    uint4 residual;
  };

  __device__ __forceinline__ float alpha() const {
    float a = 1.0f;
    if (x_scale_inv) a *= *x_scale_inv;
    if (w_scale_inv) a *= *w_scale_inv;
    return a;
  }

  __device__ __forceinline__ In load(int row, int c) const {
    In in = {};
    auto bf4 = [](const void* base, int64_t j) {
      return *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + j);
    };
    const int64_t at = int64_t(row) * N + c;
    if (bias) in.bias = bf4(bias, c);
    if (gate) in.gate = bf4(gate, int64_t(one_gate ? 0 : row / gate_rows) * N + c);
    if (!residual) return in;
    if (out_dtype == TE_BF16) {
      const uint2 r = bf4(residual, at);
      in.residual.x = r.x;
      in.residual.y = r.y;
    } else {
      in.residual = *reinterpret_cast<const uint4*>(static_cast<const float*>(residual) + at);
    }
    return in;
  }

  // out = residual_scale * residual + gate * act(alpha v + bias) at columns c .. c + 3 of a row, and z
  __device__ __forceinline__ void store(int row, int c, float alpha, float (&v)[4], const In& in) const {
    const int64_t at = int64_t(row) * N + c;
    const float bb[4] = {bf16_lo(in.bias.x), bf16_hi(in.bias.x), bf16_lo(in.bias.y), bf16_hi(in.bias.y)};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(v[k], alpha, bb[k]);
    if (z)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(z) + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    const f32x2 v01 = act2(act, f2(v[0], v[1])), v23 = act2(act, f2(v[2], v[3]));
    float o[4] = {v01.x, v01.y, v23.x, v23.y};
    if (gate) {
      o[0] *= bf16_lo(in.gate.x); o[1] *= bf16_hi(in.gate.x);
      o[2] *= bf16_lo(in.gate.y); o[3] *= bf16_hi(in.gate.y);
    }
    if (out_dtype == TE_BF16) {
      const float rr[4] = {bf16_lo(in.residual.x), bf16_hi(in.residual.x), bf16_lo(in.residual.y), bf16_hi(in.residual.y)};
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = fmaf(residual_scale, rr[k], o[k]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) =
          make_float4(fmaf(residual_scale, __uint_as_float(in.residual.x), o[0]),
                      fmaf(residual_scale, __uint_as_float(in.residual.y), o[1]),
                      fmaf(residual_scale, __uint_as_float(in.residual.z), o[2]),
                      fmaf(residual_scale, __uint_as_float(in.residual.w), o[3]));
    }
  }
};

__device__ __forceinline__ int cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return int(n);
}

// Four floats of a CTA of the cluster.  (Volatile, so that it stays behind the
// cluster's barrier, and no more, so that loads overlap.)
__device__ __forceinline__ float4 load_cluster4(uint32_t at) {
  float4 u;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w)
               : "r"(at));
  return u;
}

struct FewParams {  // aligned like its tensor maps
  CUtensorMap w;
  CUtensorMap x;
  End end;
  int M, num_kb;
  int* status;
};

// fp32 accumulator, both operands bf16 or E4M3, A (W) MN-major or, for W^T, K-major, B (x) K-major, N >> 3, M >> 4.
template <bool FP8, int NT, bool WT>
__device__ constexpr uint32_t instr_desc() {
  return (1u << 4) | ((FP8 ? 0u : 1u) << 7) | ((FP8 ? 0u : 1u) << 10) | ((WT ? 0u : 1u) << 15) | (uint32_t(NT >> 3) << 17) |
         (uint32_t(kCols >> 4) << 24);
}

template <bool FP8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (FP8)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

template <bool FP8, int NT, bool WT>
__global__ void __launch_bounds__(kThreads, 2) dense_few_kernel(const __grid_constant__ FewParams p) {
  using F = Form<FP8, NT>;
  constexpr int STAGES = F::kStages;
  constexpr uint32_t IDESC = instr_desc<FP8, NT, WT>();
  constexpr int MMA_K = 32 / (FP8 ? 1 : 2);  // K of one instruction
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(smem);
  __shared__ uint64_t full[STAGES], empty[STAGES], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = cluster_ctas(), rank = int(cluster_rank());
  const int col0 = int(blockIdx.x) / ranks * kCols;
  const int row0 = int(blockIdx.y) * NT, rows = p.M - row0 < NT ? p.M - row0 : NT;
  const int kb0 = int(int64_t(p.num_kb) * rank / ranks), kb1 = int(int64_t(p.num_kb) * (rank + 1) / ranks);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    abort_flag = 0;
    mbar_init_fence();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.x)) : "memory");
  }
  // Launched as a programmatic dependent: nothing is read before the kernel in front has finished.  Nor is
  // tensor memory taken before that, which the kernel in front may still have to allocate, and the next
  // kernel, which may take some before it waits, is let in after.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto issue = [&](int kb, int stage) {
    const uint32_t bar = smem_u32(&full[stage]);
    const uint32_t w_dst = smem_u32(smem + stage * F::kStage);
    mbar_expect_tx(bar, F::kStage);
    if constexpr (WT) {
      tma_load_2d(w_dst, &p.w, bar, kb * F::kK, col0);
    } else {
#pragma unroll
      for (int i = 0; i < kCols / F::kK; ++i)
        tma_load_2d(w_dst + i * F::kK * kRowBytes, &p.w, bar, col0 + i * F::kK, kb * F::kK);
    }
    tma_load_2d(w_dst + kWTile, &p.x, bar, kb * F::kK, row0);
  };
  const int first = kb1 - kb0 < STAGES ? kb1 - kb0 : STAGES;  // tiles that fill the ring
  if (threadIdx.x == 0)  // (its own barriers: the others have yet to see them)
    for (int s = 0; s < first; ++s) issue(kb0 + s, s);
  __syncwarp();
  if (warp == 1) tmem_alloc<1>(smem_u32(&tmem_slot), NT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, last_parity = 0;  // of the tile last brought to each stage
      for (int kb = kb0 + first; kb < kb1; ++kb) {
        if (!mbar_try_wait(smem_u32(&empty[stage]), phase) &&
            !wait_bounded(smem_u32(&empty[stage]), phase, &abort_flag, p.status, kWaitLimitNs, true))
          break;
        issue(kb, stage);
        last_parity = (last_parity & ~(1u << stage)) | ((phase ^ 1) << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      // copies in flight land before the CTA goes on (without a failure they all have)
      for (int s = 0; s < first; ++s)
        wait_bounded(smem_u32(&full[s]), (last_parity >> s) & 1, &abort_flag, p.status, kDrainLimitNs, false);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_try_wait(smem_u32(&full[stage]), phase) &&
            !wait_bounded(smem_u32(&full[stage]), phase, &abort_flag, p.status, kWaitLimitNs, true))
          break;
        tc_fence_after();
        const uint32_t w_base = smem_u32(smem + stage * F::kStage), x_base = w_base + kWTile;
#pragma unroll
        for (int j = 0; j < kRowBytes / 32; ++j)
          mma<FP8>(tmem,
                   WT ? smem_desc(w_base + j * 32, 16, 8 * kRowBytes)
                      : smem_desc(w_base + j * MMA_K * kRowBytes, F::kK * kRowBytes, 8 * kRowBytes),
                   smem_desc(x_base + j * 32, 16, 8 * kRowBytes), IDESC, (kb != kb0 || j != 0) ? 1u : 0u);
        umma_commit<1>(smem_u32(&empty[stage]));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      umma_commit<1>(smem_u32(&done));  // every MMA issued so far
      wait_bounded(smem_u32(&done), 0, &abort_flag, p.status, kWaitLimitNs, false);
    }
  } else {
    int ok = 1;
    if (lane == 0) ok = wait_bounded(smem_u32(&done), 0, &abort_flag, p.status, kWaitLimitNs, true) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) {
      while (!mbar_try_wait(smem_u32(&done), 0)) {  // it has completed: every lane observes it
      }
      __syncwarp();
      tc_fence_after();
      const int quad = warp & 3;
      // (the ring is no longer read: its copies have landed and its MMAs are done)
#pragma unroll 1
      for (int c = (warp - 2) / 4 * 32; c < NT && c < rows; c += (kThreads / 32 - 2) / 4 * 32) {
        uint32_t r[32];
        tmem_ld32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(c), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(c + j) * kPitch + quad * 32 + lane] = __uint_as_float(r[j]);
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<1>(tmem, NT);
  }
  // Four neighbouring columns of a row to a thread at a time.  What the end reads besides the sums is on its
  // way while the cluster meets, and then while the place in front is written.
  constexpr int kQuads = kCols / 4;
  static_assert(kThreads % kQuads == 0, "a thread's columns stay the same");
  const float alpha = p.end.alpha();
  const int c = int(threadIdx.x) % kQuads * 4, step = ranks * (kThreads / kQuads);
  int row = (rank * kThreads + int(threadIdx.x)) / kQuads;
  if (col0 + c >= p.end.N) row = rows;
  End::In in = {};
  if (row < rows) in = p.end.load(row0 + row, col0 + c);
  __syncwarp();
  if (ranks > 1) cluster_sync();
  {
    ClusterFlags<kMaxCluster> flags(&abort_flag, ranks, rank);
    uint32_t sums[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      sums[r] = map_to_rank(smem_u32(part + row * kPitch + c), uint32_t(r < ranks ? r : rank));
    while (row < rows) {
      float4 u[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        u[r] = r < ranks ? load_cluster4(sums[r]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        sums[r] += uint32_t(step * kPitch * sizeof(float));
      }
      float v[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int r = 1; r < kMaxCluster; ++r) {
        v[0] += u[r].x; v[1] += u[r].y; v[2] += u[r].z; v[3] += u[r].w;
      }
      if (flags.raised()) break;
      const End::In now = in;
      const int at = row0 + row;
      row += step;
      if (row < rows) in = p.end.load(row0 + row, col0 + c);
      p.end.store(at, col0 + c, alpha, v, now);
    }
  }
  __syncwarp();
  if (ranks > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// Tokens of a tile.
int tile_tokens(int64_t M) { return M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// CTAs to a tile: up to one CTA an SM in all as long as each has a stage of K, and up to two, which an SM
// holds at once, while each has 8 (in all 7 / 8 of them: clusters do not fill every SM of a GPC).  (us, two /
// one CTA an SM: [14336, 4096] in bf16 at one token 20.4 / 21.7, at 128 27.5 / 33.8; with 2 stages instead
// of 8 [2048, 4096] in E4M3 goes from 5.1 to 5.8.  [4096, 9728] in E4M3 at 128 tokens, all of two CTAs an SM /
// half of them: 26 / 21.)  Clusters of 8 on more than 3 / 4 of the SMs wait for room and want 8 stages too ([1024,
// 1024] at 256 tokens in bf16: 9.6 us, of 4 7.5; [1024, 1024] at one, on half the SMs, 4.0 and 4.6).
int cluster_of(int64_t tiles, int64_t num_kb) {
  const int64_t sms = num_sms();
  int ranks = 1;
  while (ranks < kMaxCluster && num_kb >= ranks * 2) {
    const int64_t ctas = tiles * ranks * 2;
    const bool full = ctas > sms || (ranks * 2 == kMaxCluster && ctas * 4 > sms * 3);
    if (full && (ctas * 4 > sms * 7 || num_kb < ranks * 2 * 8)) break;
    ranks *= 2;
  }
  return ranks;
}

template <bool FP8, int NT, bool WT>
te_status launch(const GemmArgs& g, cudaStream_t s) {
  using F = Form<FP8, NT>;
  static PerDevice<bool> attr_done;
  bool ok = false;
  if (!attr_done.get(&ok, [](bool* v) {
        *v = cudaFuncSetAttribute(dense_few_kernel<FP8, NT, WT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  int(F::kSmem)) == cudaSuccess;
        return *v;
      }))
    return TE_ERR_CUDA;
  FewParams p;
  memset(&p, 0, sizeof(p));
  const int dt = FP8 ? TE_E4M3 : TE_BF16;
  const bool w = WT ? make_tmap_2d(&p.w, g.B, dt, g.K, g.N, F::kK, kCols, 128)
                    : make_tmap_2d(&p.w, g.B, dt, g.N, g.K, F::kK, F::kK, 128);
  if (!w || !make_tmap_2d(&p.x, g.A, dt, g.K, g.M, F::kK, NT, 128))
    return TE_ERR_CUDA;
  p.end = End{g.a_scale_inv, g.b_scale_inv, g.bias, g.gate, g.residual, g.D, g.saved_h, g.residual_scale,
              g.cast.out_dtype, g.act, int(g.N), int(g.gate_rows), g.gate_rows == g.M};
  p.M = int(g.M);
  p.num_kb = int(ceil_div(g.K, int64_t(F::kK)));
  p.status = device_status_ptr();
  const int blocks = int(ceil_div(g.N, int64_t(kCols)));
  const int rows = int(ceil_div(g.M, int64_t(NT)));
  const int ranks = cluster_of(int64_t(blocks) * rows, p.num_kb);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks * ranks), unsigned(rows));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = F::kSmem;
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
  return cudaLaunchKernelEx(&cfg, dense_few_kernel<FP8, NT, WT>, p) == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

template <bool FP8, bool WT>
te_status launch_of(const GemmArgs& g, cudaStream_t s) {
  const int nt = tile_tokens(g.M);
  return nt == 32 ? launch<FP8, 32, WT>(g, s) : nt == 64 ? launch<FP8, 64, WT>(g, s) : launch<FP8, 128, WT>(g, s);
}

}  // namespace

// Up to 32 tokens always; up to 64 with at most 3 / 2 tiles an SM; and with more where a tile's K is split
// (half a tile an SM, or 7 / 8 with K of 16 stages).  Behind that the batch product's tiles, whose loads serve
// twice the columns, are faster.  Measured (us, here / there):
//   [14336, 4096]  128 tokens bf16 28 / 58, E4M3 20 / 43; 256: 36 / 49, 24 / 39; 512: 59 / 58, 36 / 41
//   [4096, 14336]  1: 23 / 38, 14 / 27; 64: 25 / 39, 17 / 23; 128: 31 / 42, 22 / 26
//   [4096, 28672]  1: 41 / 64, 23 / 35; 64: 43 / 45, 27 / 28; 128 (there): 57 / 49, 40 / 31
//   [4096, 57344]  1: 74 / 104, 41 / 54; 32: 81 / 86, 49 / 48
//   [1024, 1024]   1024: 13 / 15, 11 / 12;  [4096, 512]  2048: 18 / 29, 14 / 19
bool dense_few_serves(int64_t M, int64_t N, int64_t K, int ab_dtype) {
  const int nt = tile_tokens(M);
  const int64_t tiles = ceil_div(N, int64_t(kCols)) * ceil_div(M, int64_t(nt)), sms = num_sms();
  if (nt == 32 || tiles * 2 <= sms * (nt == 64 ? 3 : 1)) return true;
  return cluster_of(tiles, ceil_div(K, int64_t(kRowBytes / (ab_dtype == TE_E4M3 ? 1 : 2)))) > 1;
}

te_status launch_dense_few(const GemmArgs& g, cudaStream_t s) {
  if (g.M == 0) return TE_OK;
  const bool wt = g.epilogue == EPI_BIAS;
  if ((!wt && g.epilogue != EPI_RESIDUAL) || !g.a_kmajor || g.b_kmajor != int(wt) ||
      !dense_few_serves(g.M, g.N, g.K, g.ab_dtype))
    return TE_ERR_UNSUPPORTED;
  ProfileScope prof(wt ? TE_KERNEL_GEMM : TE_KERNEL_GEMM_ACT, s);
  if (g.ab_dtype == TE_E4M3) return wt ? launch_of<true, true>(g, s) : launch_of<true, false>(g, s);
  return wt ? launch_of<false, true>(g, s) : launch_of<false, false>(g, s);
}

}  // namespace te

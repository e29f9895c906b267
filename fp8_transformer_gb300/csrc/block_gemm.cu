// Product of two packed 4-bit operands on the tensor cores: D[M, N] = alpha * A B^T + bias with
// every block's scale applied inside tcgen05.mma (kind::mxf4, kind::mxf4nvf4).
//
// Operands lie with K inner, 256 codes to a 128-byte row of a stage, in the 128-byte swizzle that
// TMA writes.  Scales come as whole 512-byte tiles (128 rows x 4 blocks) whose byte order is that
// of tcgen05.cp.32x128b, so the MMA thread moves a tile into tensor memory with one instruction
// and no thread touches a scale.  cp and mma of one thread execute in order, so a single set of
// scale columns serves all stages.  Out-of-range codes and scales are filled with zeros by TMA,
// which is what a short last K block needs.
//
// Two forms:
//  * block_gemm_kernel, for batches of rows: persistent CTA pairs (cta_group::2) on 256 x 256
//    tiles.  The accumulator takes 256 of the 512 tensor-memory columns and the scales of a stage
//    up to 48, so there is one accumulator; the epilogue warps copy it to registers and hand it
//    back before they convert and store, so only that copy is not hidden behind the next tile.
//  * block_gemm_few_kernel, for few rows (tokens): bound by the bytes of the weights.  The
//    weights take the 128-row side of the MMA and the tokens its short side, so no tensor-core row
//    is wasted on absent tokens, and a cluster of CTAs splits K; their partial tiles are added
//    through distributed shared memory in rank order, so the result does not vary.
//
// Every wait is bounded, as in the other GEMM.
#include <cuda.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "block.cuh"
#include "kernels.h"
#include "sync.cuh"
#include "umma.cuh"

namespace te {
namespace {

constexpr int kRowBytes = 128;   // bytes of K of a tile row in a stage
constexpr int kStageK = 256;     // codes of K in a stage
constexpr int kTile = 512;       // bytes of a scale tile
constexpr int kSteps = 4;        // tcgen05.mma steps of 64 codes in a stage

// Scale tiles of a stage along K (4 blocks each).
__host__ __device__ constexpr int stage_groups(int fmt) { return kStageK / (4 * block_len(fmt)); }

// Instruction descriptor of the block-scaled kinds: E2M1 operands, N >> 3, the scales' type
// (E8M0 or E4M3), M >> 4; the scale ids (which pair of a column's bytes) are added by the step.
template <int FMT>
__device__ __forceinline__ constexpr uint32_t block_idesc(int m, int n) {
  return (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) |
         (uint32_t(FMT == TE_NVFP4 ? 0 : 1) << 23) | (uint32_t(m >> 4) << 24);
}

template <int FMT, int CG>
__device__ __forceinline__ void block_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
#define TE_BLOCK_MMA(CGS, KINDS)                                                               \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                               \
               "tcgen05.mma.cta_group::" CGS ".kind::" KINDS                                   \
               " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),                              \
               "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb))
  if constexpr (FMT == TE_NVFP4) {
    if constexpr (CG == 1) TE_BLOCK_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else TE_BLOCK_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if constexpr (CG == 1) TE_BLOCK_MMA("1", "mxf4.block_scale.scale_vec::2X");
    else TE_BLOCK_MMA("2", "mxf4.block_scale.scale_vec::2X");
  }
#undef TE_BLOCK_MMA
}

// One scale tile from shared memory into 4 tensor-memory columns (of both CTAs of a pair, each
// from its own shared memory), repeated over the four 32-lane quarters.
template <int CG>
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint32_t smem) {
  // no swizzle; core matrices of 8 rows x 16 bytes, 128 bytes apart
  const uint64_t desc = uint64_t((smem & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (1ull << 46);
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// The MMAs of one stage: copies its scales, then 4 steps.  sa / sb: the stage's scale tiles in
// shared memory, [row tiles of 128][groups]; RB: 128-row tiles of B's scales.
template <int FMT, int CG, int RB>
__device__ __forceinline__ void stage_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb,
                                          uint32_t tsa, uint32_t tsb, uint32_t idesc, bool first) {
  constexpr int G = stage_groups(FMT);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    scale_copy<CG>(tsa + g * 4, sa + g * kTile);
#pragma unroll
    for (int r = 0; r < RB; ++r) scale_copy<CG>(tsb + (g * RB + r) * 4, sb + (r * G + g) * kTile);
  }
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int g = FMT == TE_NVFP4 ? j : j / 2;                       // the step's scale tile
    const uint32_t id = FMT == TE_NVFP4 ? 0u : uint32_t(j & 1) * 2;  // and byte pair in it
    block_mma<FMT, CG>(d, smem_desc(a + j * 32, 16, 8 * kRowBytes), smem_desc(b + j * 32, 16, 8 * kRowBytes),
                       idesc | (id << 4) | (id << 29), tsa + g * 4, tsb + g * RB * 4,
                       (first && j == 0) ? 0u : 1u);
  }
}

struct BlockGemmDev {
  int64_t M, N;
  int num_m, num_n, num_kb;
  int group_m;
  const float* a_scale_inv;
  const float* b_scale_inv;
  const void* bias;
  int bias_dtype;
  void* D;
  int d_dtype;
  int b_ready;
  int* status;
};

struct BlockGemmParams {
  CUtensorMap tmA, tmB, tmSA, tmSB;
  BlockGemmDev g;
};

__device__ __forceinline__ void prefetch_maps(const BlockGemmParams& p) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmA)) : "memory");
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmB)) : "memory");
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmSA)) : "memory");
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmSB)) : "memory");
}

__device__ __forceinline__ float alpha_of(const BlockGemmDev& g) {
  float alpha = 1.0f;
  if (g.a_scale_inv) alpha *= *g.a_scale_inv;
  if (g.b_scale_inv) alpha *= *g.b_scale_inv;
  return alpha;
}

__device__ __forceinline__ float load_bias(const void* bias, int dtype, int64_t j) {
  return dtype == TE_BF16 ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(bias) + j))
                          : __ldg(static_cast<const float*>(bias) + j);
}

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return mbar_try_wait(bar, parity) || wait_bounded(bar, parity, abort_flag, status, kWaitLimitNs, true);
}

// ------------------------------------------------------------------ rows by the batch -----

constexpr int BM = 128;  // accumulator rows of a CTA
constexpr int BN = 256;  // accumulator columns
constexpr int kEpiWarps = 8;
constexpr int kBatchThreads = 32 * (2 + kEpiWarps);

template <int FMT, int CG>
struct BatchCfg {
  static constexpr int G = stage_groups(FMT);
  static constexpr int kBRows = BN / CG;
  static constexpr int kA = BM * kRowBytes;
  static constexpr int kB = kBRows * kRowBytes;
  static constexpr int kSA = G * kTile;
  static constexpr int kSB = 2 * G * kTile;  // the scales of all 256 columns, in each CTA
  static constexpr int kStage = kA + kB + kSA + kSB;
  static constexpr int kStages = (226 * 1024 - 2048) / kStage;
  static constexpr size_t kSmem = size_t(kStages) * kStage + 1024 + 256;
  static constexpr uint32_t kTsa = BN, kTsb = BN + 4 * G;  // tensor-memory columns of the scales
};

template <int FMT, int CG>
__global__ void __launch_bounds__(kBatchThreads, 1)
    block_gemm_kernel(const __grid_constant__ BlockGemmParams p) {
  using C = BatchCfg<FMT, CG>;
  constexpr int STAGES = C::kStages;
  const BlockGemmDev& g = p.g;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smA = smem_u32(smem), smB = smA + STAGES * C::kA;
  const uint32_t smSA = smB + STAGES * C::kB, smSB = smSA + STAGES * C::kSA;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStage);
  uint64_t* full = bars;
  uint64_t* empty = bars + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cluster_rank();
  const bool leader = rank == 0;
  const int cluster_id = int(blockIdx.x) / CG, num_clusters = int(gridDim.x) / CG;
  const int num_tiles = g.num_m * g.num_n;
  // raster groups of group_m m-tiles, m fastest: a group's A stays in L2 while it sweeps B
  auto tile_of = [&](int t, int& tm, int& tn) {
    const int size = g.group_m * g.num_n, first = t / size * g.group_m, in = t % size;
    const int gm = min(g.num_m - first, g.group_m);
    tm = first + in % gm;
    tn = in / gm;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(tempty), 32 * kEpiWarps * CG);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    mbar_init_fence();
    prefetch_maps(p);
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the peer's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;
      bool ok = true;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        int tm, tn;
        tile_of(t, tm, tn);
        const int mt = tm * CG + int(rank);  // this CTA's 128 rows
        for (int kb = 0; kb < g.num_kb; ++kb) {
          if (!wait_or_abort(smem_u32(&empty[stage]), phase ^ 1, abort_flag, g.status)) {
            ok = false;
            break;
          }
          const uint32_t fb = CG == 1 ? smem_u32(&full[stage]) : map_to_rank(smem_u32(&full[stage]), 0);
          if (leader) mbar_expect_tx(smem_u32(&full[stage]), CG * C::kStage);
          auto load = [&](uint32_t dst, const CUtensorMap* m, int c0, int c1) {
            if constexpr (CG == 1) tma_load_2d(dst, m, fb, c0, c1);
            else tma_load_2d_pair(dst, m, fb, c0, c1);
          };
          load(smA + stage * C::kA, &p.tmA, kb * kRowBytes, mt * BM);
          load(smB + stage * C::kB, &p.tmB, kb * kRowBytes, tn * BN + int(rank) * C::kBRows);
          load(smSA + stage * C::kSA, &p.tmSA, kb * C::G * 64, mt);
          load(smSB + stage * C::kSB, &p.tmSB, kb * C::G * 64, tn * 2);
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (leader) {
        // copies still in flight (the pair's) complete before the CTAs may exit
        for (int s = 0; s < STAGES; ++s)
          if (issued & (1u << s))
            wait_bounded(smem_u32(&full[s]), (last_parity >> s) & 1, abort_flag, g.status, kDrainLimitNs, false);
      } else if (!ok) {
        // the peer's copies signal the leader: after an abort give them time to land
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 100000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = block_idesc<FMT>(BM * CG, BN);
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, acc_phase ^= 1) {
        if (!wait_or_abort(smem_u32(tempty), acc_phase ^ 1, abort_flag, g.status)) break;
        tc_fence_after();
        for (int kb = 0; kb < g.num_kb; ++kb) {
          if (!wait_or_abort(smem_u32(&full[stage]), phase, abort_flag, g.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          stage_mma<FMT, CG, 2>(tmem, smA + stage * C::kA, smB + stage * C::kB, smSA + stage * C::kSA,
                                smSB + stage * C::kSB, tmem + C::kTsa, tmem + C::kTsb, idesc, kb == 0);
          if constexpr (CG == 1) umma_commit<1>(smem_u32(&empty[stage]));
          else umma_commit_mc(smem_u32(&empty[stage]), 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (CG == 1) umma_commit<1>(smem_u32(tfull));
        else umma_commit_mc(smem_u32(tfull), 0x3);
      }
      // own MMAs complete before tensor memory is released
      umma_commit<CG>(smem_u32(drain));
      wait_bounded(smem_u32(drain), 0, abort_flag, g.status, kDrainLimitNs, false);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const float alpha = alpha_of(g);
    const uint32_t tempty_leader = CG == 1 ? smem_u32(tempty) : map_to_rank(smem_u32(tempty), 0);
    uint32_t phase = 0;
    for (int t = cluster_id; t < num_tiles; t += num_clusters, phase ^= 1) {
      int ok = 1;
      if (lane == 0) ok = wait_bounded(smem_u32(tfull), phase, abort_flag, g.status, kWaitLimitNs, true) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      // the phase has completed; every lane observes it before touching tensor memory
      while (!mbar_try_wait(smem_u32(tfull), phase)) {
      }
      __syncwarp();
      tc_fence_after();
      int tm, tn;
      tile_of(t, tm, tn);
      const int64_t row = (int64_t(tm) * CG + rank) * BM + quad * 32 + lane;
      const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + uint32_t(half * (BN / 2));
      // this warp's half of the columns into registers, then the accumulator is free
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(taddr + c * 32, r[c]);
      tmem_ld_wait();
      tc_fence_before();
      if constexpr (CG == 1) mbar_arrive(tempty_leader);
      else mbar_arrive_cluster(tempty_leader);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t col0 = int64_t(tn) * BN + half * (BN / 2) + c * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 8 columns at a time; N is a multiple of 16
          const int64_t col = col0 + q * 8;
          if (row < g.M && col < g.N) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float b = g.bias ? load_bias(g.bias, g.bias_dtype, col + i) : 0.0f;
              v[i] = fmaf(__uint_as_float(r[c][q * 8 + i]), alpha, b);
            }
            const int64_t at = row * g.N + col;
            if (g.d_dtype == TE_F32) {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.D) + at);
              o[0] = make_float4(v[0], v[1], v[2], v[3]);
              o[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.D) + at) =
                  make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7]));
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // no MMA of the pair still writes this CTA's columns
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<CG>(tmem, 512);
  }
}

// ------------------------------------------------------------------ few rows --------------

constexpr int kFewThreads = 192;  // producer, MMA, four epilogue warps

template <int FMT, int TOK>
struct FewCfg {
  static constexpr int G = stage_groups(FMT);
  static constexpr int kW = BM * kRowBytes;   // 128 weight rows
  static constexpr int kT = TOK * kRowBytes;  // the tokens
  static constexpr int kS = G * kTile;        // scales of either (tokens: one tile of 128 rows)
  static constexpr int kStage = kW + kT + 2 * kS;
  static constexpr int kStages = (200 * 1024) / kStage < 10 ? (200 * 1024) / kStage : 10;
  static constexpr size_t kSmem = size_t(kStages) * kStage + 1024 + 256;
  static constexpr uint32_t kTsw = TOK < 32 ? 32 : TOK, kTst = kTsw + 4 * G;
  static constexpr uint32_t kNeed = kTst + 4 * G;
  static constexpr uint32_t kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : 256;
  static_assert(kNeed <= 256 && kStages * kStage >= BM * TOK * 4, "columns; room for the partial tile");
};

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void store_one(const BlockGemmDev& g, int64_t at, float v) {
  if (g.d_dtype == TE_F32) static_cast<float*>(g.D)[at] = v;
  else static_cast<__nv_bfloat16*>(g.D)[at] = __float2bfloat16_rn(v);
}

// Grid: (clusters of `split` CTAs along K) x tiles of 128 weight rows; M <= TOK tokens.  Here the
// MMA's A side is the weights (g's B operand).
template <int FMT, int TOK>
__global__ void __launch_bounds__(kFewThreads, 1)
    block_gemm_few_kernel(const __grid_constant__ BlockGemmParams p, int split) {
  using C = FewCfg<FMT, TOK>;
  constexpr int STAGES = C::kStages;
  const BlockGemmDev& g = p.g;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smW = smem_u32(smem), smT = smW + STAGES * C::kW;
  const uint32_t smSW = smT + STAGES * C::kT, smST = smSW + STAGES * C::kS;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStage);
  uint64_t* full = bars;
  uint64_t* empty = bars + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(blockIdx.x) % split, tile = int(blockIdx.x) / split;
  const int kb0 = int(int64_t(g.num_kb) * rank / split), kb1 = int(int64_t(g.num_kb) * (rank + 1) / split);
  const int nkb = kb1 - kb0;  // at least 1: split <= num_kb

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    mbar_init_fence();
    prefetch_maps(p);
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      auto load_w = [&](int stage, int kb) {
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_expect_tx(fb, C::kStage);
        tma_load_2d(smW + stage * C::kW, &p.tmB, fb, kb * kRowBytes, tile * BM);
        tma_load_2d(smSW + stage * C::kS, &p.tmSB, fb, kb * C::G * 64, tile);
      };
      auto load_t = [&](int stage, int kb) {
        const uint32_t fb = smem_u32(&full[stage]);
        tma_load_2d(smT + stage * C::kT, &p.tmA, fb, kb * kRowBytes, 0);
        tma_load_2d(smST + stage * C::kS, &p.tmSA, fb, kb * C::G * 64, 0);
      };
      // the weights of the first stages may be on their way before the kernel that packs the
      // tokens is done
      int early = 0;
      if (g.b_ready)
        for (; early < nkb && early < STAGES; ++early) load_w(early, kb0 + early);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int i = 0; i < nkb; ++i) {
        if (!wait_or_abort(smem_u32(&empty[stage]), phase ^ 1, abort_flag, g.status)) break;
        if (i >= early) load_w(stage, kb0 + i);
        load_t(stage, kb0 + i);
        issued = i + 1;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      // after an abort: copies still in flight land before the CTA may exit (the early ones of
      // stages that no token load followed cannot be waited for; give them time)
      for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        wait_bounded(smem_u32(&full[i % STAGES]), (i / STAGES) & 1, abort_flag, g.status, kDrainLimitNs, false);
      if (issued < early) {
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 100000ull) {
        }
      }
    }
  } else if (warp == 1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (lane == 0) {
      constexpr uint32_t idesc = block_idesc<FMT>(BM, TOK);
      int stage = 0;
      uint32_t phase = 0;
      for (int i = 0; i < nkb; ++i) {
        if (!wait_or_abort(smem_u32(&full[stage]), phase, abort_flag, g.status)) break;
        tc_fence_after();
        stage_mma<FMT, 1, 1>(tmem, smW + stage * C::kW, smT + stage * C::kT, smSW + stage * C::kS,
                             smST + stage * C::kS, tmem + C::kTsw, tmem + C::kTst, idesc, i == 0);
        umma_commit<1>(smem_u32(&empty[stage]));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      umma_commit<1>(smem_u32(done));
      wait_bounded(smem_u32(done), 0, abort_flag, g.status, kDrainLimitNs, false);
    }
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quad = warp & 3, row = quad * 32 + lane;
    const int64_t n = int64_t(tile) * BM + row;
    const float alpha = alpha_of(g);
    const float bias = (g.bias && n < g.N) ? load_bias(g.bias, g.bias_dtype, n) : 0.0f;
    const int tokens = int(g.M);
    int ok = 1;
    if (lane == 0) ok = wait_bounded(smem_u32(done), 0, abort_flag, g.status, kWaitLimitNs, true) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) {
      while (!mbar_try_wait(smem_u32(done), 0)) {
      }
      __syncwarp();
    }
    tc_fence_after();
    // the partial tile, [token][128 rows] fp32, over the pipeline's buffers: every stage has been
    // consumed (`done` follows the last MMA)
    float* part = reinterpret_cast<float*>(smem);
    const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < (TOK + 31) / 32; ++c) {
      uint32_t r[32];
      tmem_ld32(taddr + c * 32, r);
      tmem_ld_wait();
      if (!ok) break;
      if (split == 1) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i < tokens && n < g.N)
            store_one(g, int64_t(c * 32 + i) * g.N + n, fmaf(__uint_as_float(r[i]), alpha, bias));
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i < TOK) part[(c * 32 + i) * BM + row] = __uint_as_float(r[i]);
      }
    }
    tc_fence_before();
    if (split > 1) {
      cluster_sync();
      // tokens go round the ranks; each sums its tokens' columns in rank order
      if (ok)
        for (int t = rank; t < tokens; t += split) {
          const uint32_t at = smem_u32(part + t * BM + row);
          float s = 0.0f;
          for (int k = 0; k < split; ++k) s += ld_cluster(map_to_rank(at, uint32_t(k)));
          if (n < g.N) store_one(g, int64_t(t) * g.N + n, fmaf(s, alpha, bias));
        }
    }
  }
  if (split > 1) {
    if (warp < 2) {
      __syncwarp();
      cluster_sync();  // the partial tiles are written
    }
    __syncwarp();
    cluster_sync();  // and read, before any CTA of the cluster exits
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<1>(tmem, C::kCols);
  }
}

// ------------------------------------------------------------------ host side -------------

template <class Kernel>
te_status launch_clusters(Kernel kernel, int grid, int threads, size_t smem, int cluster, cudaStream_t s,
                          const BlockGemmParams& prm, int split) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster == 1 ? 1 : 2;
  cudaError_t e;
  if constexpr (std::is_invocable_v<Kernel, BlockGemmParams, int>) e = cudaLaunchKernelEx(&cfg, kernel, prm, split);
  else e = cudaLaunchKernelEx(&cfg, kernel, prm);
  if (e != cudaSuccess) return TE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

template <class Kernel>
bool allow_smem(Kernel kernel, size_t smem, PerDevice<bool>& set) {
  bool ok = false;
  return set.get(&ok, [&](bool* v) {
    *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) == cudaSuccess;
    return *v;
  });
}

// Codes as bytes: 128-byte rows of 256 codes, `rows` rows to a box.
bool code_map(CUtensorMap* tm, const void* ptr, int64_t rows, int64_t K, uint32_t box_rows) {
  return make_tmap_2d(tm, ptr, TE_E4M3, uint64_t(K / 2), uint64_t(rows), kRowBytes, box_rows, true);
}

template <int FMT, int CG>
te_status launch_batch(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  using C = BatchCfg<FMT, CG>;
  BlockGemmDev& g = prm.g;
  const uint64_t groups = uint64_t(scale_groups(FMT, a.K));
  g.num_m = int(ceil_div(a.M, BM * CG));
  g.num_n = int(ceil_div(a.N, BN));
  if (!code_map(&prm.tmA, a.A, a.M, a.K, BM) || !code_map(&prm.tmB, a.B, a.N, a.K, C::kBRows) ||
      !make_tmap_scales(&prm.tmSA, a.a_scales, groups, uint64_t(ceil_div(a.M, 128)), C::G, 1) ||
      !make_tmap_scales(&prm.tmSB, a.b_scales, groups, uint64_t(ceil_div(a.N, 128)), C::G, 2))
    return TE_ERR_CUDA;
  const int64_t tile_bytes = int64_t(BM) * CG * a.K / 2;
  const int64_t gm = (48ll << 20) / tile_bytes;  // A rows that a raster group may keep in L2
  g.group_m = int(gm < 4 ? 4 : gm < g.num_m ? gm : g.num_m);
  const int64_t tiles = int64_t(g.num_m) * g.num_n, slots = num_sms() / CG;
  if (tiles > 0x3fffffff) return TE_ERR_UNSUPPORTED;
  static PerDevice<bool> set;
  if (!allow_smem(block_gemm_kernel<FMT, CG>, C::kSmem, set)) return TE_ERR_CUDA;
  return launch_clusters(block_gemm_kernel<FMT, CG>, int(tiles < slots ? tiles : slots) * CG, kBatchThreads,
                         C::kSmem, CG, s, prm, 0);
}

template <int FMT, int TOK>
te_status launch_few(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  using C = FewCfg<FMT, TOK>;
  const uint64_t groups = uint64_t(scale_groups(FMT, a.K));
  if (!code_map(&prm.tmA, a.A, a.M, a.K, TOK) || !code_map(&prm.tmB, a.B, a.N, a.K, BM) ||
      !make_tmap_scales(&prm.tmSA, a.a_scales, groups, 1, C::G, 1) ||
      !make_tmap_scales(&prm.tmSB, a.b_scales, groups, uint64_t(ceil_div(a.N, 128)), C::G, 1))
    return TE_ERR_CUDA;
  const int64_t tiles = ceil_div(a.N, BM);
  if (tiles > 0x0fffffff) return TE_ERR_UNSUPPORTED;
  // K is split while the SMs outnumber the tiles and every CTA keeps two stages of K
  int split = 1;
  while (split < 8 && tiles * split * 2 <= num_sms() && split * 4 <= prm.g.num_kb) split *= 2;
  static PerDevice<bool> set;
  if (!allow_smem(block_gemm_few_kernel<FMT, TOK>, C::kSmem, set)) return TE_ERR_CUDA;
  return launch_clusters(block_gemm_few_kernel<FMT, TOK>, int(tiles) * split, kFewThreads, C::kSmem, split, s,
                         prm, split);
}

template <int FMT>
te_status launch_fmt(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  if (a.M <= 16) return launch_few<FMT, 16>(a, prm, s);
  if (a.M <= 32) return launch_few<FMT, 32>(a, prm, s);
  if (a.M <= 64) return launch_few<FMT, 64>(a, prm, s);
  if (a.M <= 128) return launch_few<FMT, 128>(a, prm, s);
  return launch_batch<FMT, 2>(a, prm, s);
}

}  // namespace

te_status launch_block_gemm(const BlockGemmArgs& a, cudaStream_t s) {
  if (a.M == 0 || a.N == 0) return TE_OK;
  BlockGemmParams prm;
  memset(&prm, 0, sizeof(prm));
  BlockGemmDev& g = prm.g;
  if (a.M > 0x7fffffff || a.N > 0x7fffffff || a.K > 0x7fffffff) return TE_ERR_UNSUPPORTED;
  g.M = a.M;
  g.N = a.N;
  g.num_kb = int(ceil_div(a.K, kStageK));
  g.a_scale_inv = a.a_scale_inv;
  g.b_scale_inv = a.b_scale_inv;
  g.bias = a.bias;
  g.bias_dtype = a.bias_dtype;
  g.D = a.D;
  g.d_dtype = a.d_dtype;
  g.b_ready = a.b_ready;
  g.status = device_status_ptr();
  ProfileScope prof(TE_KERNEL_GEMM, s);
  return a.fmt == TE_NVFP4 ? launch_fmt<TE_NVFP4>(a, prm, s) : launch_fmt<TE_MXFP4>(a, prm, s);
}

}  // namespace te

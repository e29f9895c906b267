// Product of two packed 4-bit operands on the tensor cores: D[M, N] = alpha * A B^T + bias with
// every block's scale applied inside tcgen05.mma (kind::mxf4, kind::mxf4nvf4).
//
// Operands lie with K inner, 256 codes to a 128-byte row of a stage, in the 128-byte swizzle that
// TMA writes.  Scales come as whole 512-byte tiles (128 rows x 4 blocks) in the byte order of
// tcgen05.cp.32x128b.  Out-of-range codes and scales are filled with zeros by TMA, which is what a
// short last K block needs.
//
// Two forms:
//  * block_gemm_kernel, for batches of rows: persistent CTA pairs (cta_group::2) on 256 x 256
//    tiles, 15 warps a CTA:
//      warp 0       TMA producer of the codes, five or six stages
//      warp 1       MMA issuer (in the pair's even CTA): the warp walks its loop, one lane issues
//      warps 2-9    epilogue: accumulator -> registers (rounded) -> a swizzled stage -> TMA store
//      warps 10-13  scales: from shared memory to each stage's set of tensor-memory columns, one
//                   16-byte row of a scale tile a lane.  With tcgen05.cp, 8192 x 28672 x 4096 took 453 us in
//                   MXFP4 and 588 in NVFP4 from the MMA thread, 402 and 450 from another.
//      warp 14      TMA producer of the scales
//    The accumulator takes 256 of the 512 tensor-memory columns and the scales 24 or 48 a stage, so
//    there is one accumulator, and its hand-over is not hidden: over nine tiles a pair, a tile
//    takes 1.11 us for 1024 codes of K and 1.5 us more (start and end of the launch among them).
//    Bound by the tensor pipe at 64 codes a step and, in long runs, by the power cap:
//    8192 x 28672 x 4096 takes 256 to 264 us in MXFP4 (7.4 PFLOP/s; 280 to 290 sustained), 272 to 282 in NVFP4
//    (320 sustained).  The tensor pipe is active 79% and 77% of the time.
//  * block_gemm_few_kernel, for few rows (tokens): bound by the bytes of the weights.  The
//    weights take the 128-row side of the MMA and the tokens its short side, so no tensor-core row
//    is wasted on absent tokens, and a cluster of CTAs splits K; their partial sums are
//    added through distributed shared memory in rank order, so the result does not vary.  Up to 8
//    tokens are packed here too.  One token on [28672, 4096] in MXFP4: 12.2 us, 5.1 TB/s; 33 tokens on
//    [4096, 14336] in NVFP4: 8.9 us and 2.9 for their packing.  Here tcgen05.cp does for the scales:
//    what it takes is hidden behind the weights.
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

// One scale tile from shared memory into 4 tensor-memory columns, repeated over the four 32-lane
// quarters.
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint32_t smem) {
  // no swizzle; core matrices of 8 rows x 16 bytes, 128 bytes apart
  const uint64_t desc = uint64_t((smem & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Copies a stage's scales to tensor memory.  sa / sb: its scale tiles in shared memory.
template <int FMT>
__device__ __forceinline__ void stage_scales(uint32_t sa, uint32_t sb, uint32_t tsa, uint32_t tsb) {
  constexpr int G = stage_groups(FMT);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    scale_copy(tsa + g * 4, sa + g * kTile);
    scale_copy(tsb + g * 4, sb + g * kTile);
  }
}

// The MMAs of one stage, 4 steps of 64 codes.  RB: 128-row tiles of B's scales.
template <int FMT, int CG, int RB>
__device__ __forceinline__ void stage_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t tsa, uint32_t tsb,
                                          uint32_t idesc, bool first) {
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
  int64_t M, N, K;
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
  CUtensorMap tmD;  // output boxes of 32 rows x 64 bytes (rows by the batch)
  BlockGemmDev g;
  BlockQuantArgs q;  // few rows packed inside the kernel: x and its tensor scale
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

// By ordinary loads: the bias may come from the kernel before.
__device__ __forceinline__ float load_bias(const void* bias, int dtype, int64_t j) {
  return dtype == TE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[j])
                          : static_cast<const float*>(bias)[j];
}

// r (32 consecutive columns) times alpha plus their bias, of which lane i of the warp holds column i's.
__device__ __forceinline__ void scale_and_bias(float alpha, bool have_bias, float bias, uint32_t (&r)[32]) {
  if (have_bias) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      r[i] = __float_as_uint(fmaf(__uint_as_float(r[i]), alpha, __shfl_sync(0xffffffffu, bias, i)));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
  }
}

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return mbar_try_wait(bar, parity) || wait_bounded(bar, parity, abort_flag, status, kWaitLimitNs, true);
}

// Arrives at a barrier of the pair without ordering this thread's memory accesses: what these
// signals hand over is tensor memory, whose accesses tcgen05.wait and the tcgen05 fences order: the
// arriving warp waits for its tcgen05.ld or st and fences before it, and the MMA warp, the only one to act
// on these phases, fences after its wait.  A release at cluster scope waits for the thread's global
// stores as well; it made an epilogue or scale warp's turn about 0.7 us longer.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// All lanes of a warp wait for the phase; false after an abort.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_or_abort(bar, parity, abort_flag, status) ? 1 : 0;
  if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
  // The phase that one lane saw complete stays so until this warp signals: each lane sees it itself, on
  // its first tries (in line: through the bounded wait's call, products took 1% more).  A lane that did
  // not raises the flag and records the timeout as that wait does.
  bool seen = false;
  for (int i = 0; i < 1024 && !seen; ++i) seen = mbar_try_wait(bar, parity);
  if (!seen) {
    if (status) atomicCAS(status, 0, int(TE_ERR_TIMEOUT));
    *abort_flag = 1;
  }
  return __all_sync(0xffffffffu, seen);
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Four consecutive columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint4 v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// tcgen05.wait::ld tied to the registers of the load it is for, so that no use moves above it.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// A tile from shared to global memory by the TMA engine (rows and columns past the end are left
// out), and the waits for its reads and for all of it.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ------------------------------------------------------------------ rows by the batch -----

constexpr int BM = 128;  // accumulator rows of a CTA
constexpr int BN = 256;  // accumulator columns
constexpr int kOutRow = 64;  // bytes of a row of an output stage (32 bf16 or 16 fp32 columns)
constexpr int kEpiWarps = 8;
constexpr int kScaleWarps = 4;
constexpr int kScaleProducer = 2 + kEpiWarps + kScaleWarps;  // the warp that loads the scales
constexpr int kBatchThreads = 32 * (kScaleProducer + 1);

template <int FMT>
struct BatchCfg {
  static constexpr int G = stage_groups(FMT);
  static constexpr int kBRows = BN / 2;              // B rows that a CTA holds
  static constexpr int kA = BM * kRowBytes;
  static constexpr int kB = kBRows * kRowBytes;
  static constexpr int kSA = G * kTile;
  static constexpr int kSB = 2 * G * kTile;          // the scales of all 256 columns, in each CTA
  static constexpr int kOut = 32 * kOutRow;          // an epilogue warp's output stage: 32 rows
  // Codes and scales have rings of their own.  A stage of either comes round again after its
  // release, a TMA load and its use, about 1.7 us, in which the tensor cores want five of them.
  static constexpr int kStages = FMT == TE_NVFP4 ? 5 : 6;
  static constexpr int kScaleStages = FMT == TE_NVFP4 ? 7 : 5;
  static constexpr int kBytes = kStages * (kA + kB) + kEpiWarps * kOut + kScaleStages * (kSA + kSB);
  static constexpr size_t kSmem = size_t(kBytes) + 1024 + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // tensor-memory columns of the scales: for each stage a set of A's (4 G) and B's (8 G)
  static constexpr uint32_t kSet = 12 * G;
  static_assert(BN + kStages * kSet <= 512, "tensor memory");
};

template <int FMT>
__global__ void __launch_bounds__(kBatchThreads, 1)
    block_gemm_kernel(const __grid_constant__ BlockGemmParams p) {
  using C = BatchCfg<FMT>;
  constexpr int STAGES = C::kStages, SSTAGES = C::kScaleStages;
  const BlockGemmDev& g = p.g;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smA = smem_u32(smem), smB = smA + STAGES * C::kA;
  const uint32_t smOut = smB + STAGES * C::kB;
  const uint32_t smSA = smOut + kEpiWarps * C::kOut, smSB = smSA + SSTAGES * C::kSA;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBytes);
  uint64_t* full = bars;              // a stage's codes and scale columns, both CTAs' (even CTA)
  uint64_t* empty = full + STAGES;    // the pair has consumed the stage and its scale columns
  uint64_t* sload = empty + STAGES;   // scales of a scale stage, this CTA's
  uint64_t* sempty = sload + SSTAGES;
  uint64_t* tfull = sempty + SSTAGES;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int cluster_id = int(blockIdx.x) / 2, num_clusters = int(gridDim.x) / 2;
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
      mbar_init(smem_u32(&full[s]), 1 + 2 * kScaleWarps);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int s = 0; s < SSTAGES; ++s) {
      mbar_init(smem_u32(&sload[s]), 1);
      mbar_init(smem_u32(&sempty[s]), kScaleWarps);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(tempty), 2 * kEpiWarps);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    mbar_init_fence();
    prefetch_maps(p);
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer ----------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;
      bool ok = true;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        int tm, tn;
        tile_of(t, tm, tn);
        const int mt = tm * 2 + int(rank);  // this CTA's 128 rows
        for (int kb = 0; kb < g.num_kb; ++kb) {
          if (!wait_or_abort(smem_u32(&empty[stage]), phase ^ 1, abort_flag, g.status)) {
            ok = false;
            break;
          }
          const uint32_t fb = map_to_rank(smem_u32(&full[stage]), 0);
          if (leader) mbar_expect_tx(smem_u32(&full[stage]), 2 * (C::kA + C::kB));
          tma_load_2d_pair(smA + stage * C::kA, &p.tmA, fb, kb * kRowBytes, mt * BM);
          tma_load_2d_pair(smB + stage * C::kB, &p.tmB, fb, kb * kRowBytes, tn * BN + int(rank) * C::kBRows);
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // copies still in flight into this CTA, and the peer's signals to it, come before it may exit
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) {
          const uint32_t parity = (last_parity >> s) & 1;
          if (leader) wait_bounded(smem_u32(&full[s]), parity, abort_flag, g.status, kDrainLimitNs, false);
          if (ok) wait_bounded(smem_u32(&empty[s]), parity, abort_flag, g.status, kWaitLimitNs, true);
        }
      if (!ok) {
        // after an abort: copies that the peer issued or observes get time to land
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 100000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer ------------
    // The whole warp walks the loop, so that descriptors and addresses stay in uniform registers, and
    // one elected lane issues.
    if (leader) {
      constexpr uint32_t idesc = block_idesc<FMT>(2 * BM, BN);
      const bool issuer = elect_one();
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, acc_phase ^= 1) {
        // the accumulator has been read by both CTAs: their relaxed arrivals and this fence order that
        if (!warp_wait(smem_u32(tempty), acc_phase ^ 1, abort_flag, g.status)) break;
        tc_fence_after();
        for (int kb = 0; kb < g.num_kb; ++kb) {
          // codes have landed (TMA's own signal) and the scale warps' stores are done (relaxed arrivals,
          // ordered by this fence)
          if (!warp_wait(smem_u32(&full[stage]), phase, abort_flag, g.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ts = tmem + BN + stage * C::kSet;
          if (issuer) {
            stage_mma<FMT, 2, 2>(tmem, smA + stage * C::kA, smB + stage * C::kB, ts, ts + 4 * C::G, idesc, kb == 0);
            umma_commit_mc(smem_u32(&empty[stage]), 0x3);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (issuer) umma_commit_mc(smem_u32(tfull), 0x3);
        __syncwarp();
      }
      // own MMAs complete before tensor memory is released
      if (issuer) {
        umma_commit<2>(smem_u32(drain));
        wait_bounded(smem_u32(drain), 0, abort_flag, g.status, kDrainLimitNs, false);
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------- epilogue --------------
    // Warp w takes the lanes of quadrant w % 4 and 128 of the columns.  Results go through a
    // swizzled stage of 32 rows x 64 bytes and a TMA store: from registers, with a row a thread, the
    // stores of a tile took 5 us, more than the MMAs of a tile with K = 2048.
    const int quad = warp & 3, cols = (warp - 2) >> 2;
    const float alpha = alpha_of(g);
    const uint32_t tempty_leader = map_to_rank(smem_u32(tempty), 0);
    const uint32_t out = smOut + (warp - 2) * C::kOut + lane * kOutRow;
    auto stage16 = [&](int j, const uint32_t* w) {  // 16 bytes to place j of this thread's row
      st_shared16(out + ((j ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
    };
    uint32_t phase = 0;
    for (int t = cluster_id; t < num_tiles; t += num_clusters, phase ^= 1) {
      int tm, tn;
      tile_of(t, tm, tn);
      const int row0 = (tm * 2 + int(rank)) * BM + quad * 32, col0 = tn * BN + cols * (BN / 2);
      float bias[4] = {};  // of columns col0 + 32 c + lane, under way while the MMAs run
      if (g.bias)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col0 + c * 32 + lane < g.N) bias[c] = load_bias(g.bias, g.bias_dtype, col0 + c * 32 + lane);
      if (!warp_wait(smem_u32(tfull), phase, abort_flag, g.status)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + uint32_t(cols * (BN / 2));
      auto free_accumulator = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader);
      };
      auto send = [&](int col) {  // the stage, complete, to column `col` on
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < g.M && col < g.N)
          tma_store_2d(&p.tmD, smOut + (warp - 2) * C::kOut, col, row0);
      };
      auto recycle = [&]() {  // the stage's last contents have been read
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
      };
      if (g.d_dtype == TE_F32) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(taddr + c * 32, r);
          tmem_ld_wait32(r);
          if (c == 3) free_accumulator();
          scale_and_bias(alpha, g.bias != nullptr, c == 0 ? bias[0] : c == 1 ? bias[1] : c == 2 ? bias[2] : bias[3], r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            recycle();
#pragma unroll
            for (int j = 0; j < 4; ++j) stage16(j, r + 16 * h + 4 * j);
            send(col0 + c * 32 + h * 16);
          }
        }
      } else {
        // rounded to registers, so that the accumulator is free before anything waits for a store
        uint32_t r[2][32], w[4][16];
        tmem_ld32(taddr, r[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait32(r[c & 1]);
          if (c < 3) tmem_ld32(taddr + (c + 1) * 32, r[(c + 1) & 1]);
          else free_accumulator();
          scale_and_bias(alpha, g.bias != nullptr, bias[c], r[c & 1]);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[c][i] = pack_bf16x2(__uint_as_float(r[c & 1][2 * i]), __uint_as_float(r[c & 1][2 * i + 1]));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          recycle();
#pragma unroll
          for (int j = 0; j < 4; ++j) stage16(j, w[c] + 4 * j);
          send(col0 + c * 32);
        }
      }
    }
    if (lane == 0) tma_store_wait();
  } else if (warp == kScaleProducer) {
    // ------------------------------------------------------------- scale producer --------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;
      bool ok = true;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        int tm, tn;
        tile_of(t, tm, tn);
        for (int kb = 0; kb < g.num_kb; ++kb) {
          if (!wait_or_abort(smem_u32(&sempty[stage]), phase ^ 1, abort_flag, g.status)) {
            ok = false;
            break;
          }
          const uint32_t sb = smem_u32(&sload[stage]);
          mbar_expect_tx(sb, C::kSA + C::kSB);
          tma_load_2d(smSA + stage * C::kSA, &p.tmSA, sb, kb * C::G * 64, tm * 2 + int(rank));
          tma_load_2d(smSB + stage * C::kSB, &p.tmSB, sb, kb * C::G * 64, tn * 2);
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == SSTAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      for (int s = 0; s < SSTAGES; ++s)  // copies in flight land before the CTA may exit
        if (issued & (1u << s))
          wait_bounded(smem_u32(&sload[s]), (last_parity >> s) & 1, abort_flag, g.status, kDrainLimitNs, false);
    }
  } else {
    // ------------------------------------------------------------- scales ----------------
    // Every warp writes its 32 lanes of a set: lane r takes the 16 bytes of row r of each tile.
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    int stage = 0, sstage = 0;
    uint32_t phase = 0, sphase = 0;
    bool ok = true;
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters)
      for (int kb = 0; kb < g.num_kb; ++kb) {
        if (!warp_wait(smem_u32(&sload[sstage]), sphase, abort_flag, g.status)) {
          ok = false;
          break;
        }
        const uint32_t sa = smSA + sstage * C::kSA + lane * 16, sb = smSB + sstage * C::kSB + lane * 16;
        uint4 v[3 * C::G];  // in the order of the set's columns: A's tiles, B's by block and row tile
#pragma unroll
        for (int q = 0; q < C::G; ++q) {
          v[q] = ld_shared16(sa + q * kTile);
#pragma unroll
          for (int r = 0; r < 2; ++r) v[C::G + q * 2 + r] = ld_shared16(sb + (r * C::G + q) * kTile);
        }
        // the set's last MMAs are done
        if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1, abort_flag, g.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ts = tmem + lanes + BN + stage * C::kSet;
#pragma unroll
        for (int q = 0; q < 3 * C::G; ++q) tmem_st4(ts + q * 4, v[q]);
        __syncwarp();  // every lane has read its rows
        if (lane == 0) mbar_arrive(smem_u32(&sempty[sstage]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(&full[stage]), 0));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
        if (++sstage == SSTAGES) {
          sstage = 0;
          sphase ^= 1;
        }
      }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no MMA of the pair still writes this CTA's columns, no copy its memory
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
}

// ------------------------------------------------------------------ few rows --------------

constexpr int kFewThreads = 192;  // producer, MMA, four epilogue warps

constexpr int kMaxSplit = 8;  // CTAs of a cluster that share a tile's K

template <int FMT, int TOK>
struct FewCfg {
  static constexpr int G = stage_groups(FMT);
  static constexpr int kW = BM * kRowBytes;   // 128 weight rows
  static constexpr int kT = TOK * kRowBytes;  // the tokens
  static constexpr int kS = G * kTile;        // scales of either (tokens: one tile of 128 rows)
  static constexpr int kStage = kW + kT + 2 * kS;
  // two CTAs to an SM, so that the tiles of a wide weight are all resident at once
  static constexpr int kStages = (113 * 1024 - 1024 - 256) / kStage;
  static constexpr size_t kSmem = size_t(kStages) * kStage + 1024 + 256;
  static constexpr uint32_t kTsw = TOK < 32 ? 32 : TOK, kTst = kTsw + 4 * G;
  static constexpr uint32_t kNeed = kTst + 4 * G;
  static constexpr uint32_t kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : 256;
  static_assert(kNeed <= 256 && kStages * kStage >= BM * TOK * 4, "columns; room for the partial tile");
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Four neighbouring outputs of one token (those past N left out).
__device__ __forceinline__ void store_four(const BlockGemmDev& g, int64_t token, int64_t n, const float (&v)[4]) {
  if (n >= g.N) return;  // N is a multiple of 16
  const int64_t at = token * g.N + n;
  if (g.d_dtype == TE_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(g.D) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.D) + at) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// Grid: (clusters of `split` CTAs along K) x tiles of 128 weight rows; M <= TOK tokens.  Here the
// MMA's A side is the weights (g's B operand).  Rank t % split adds up token t: it reads the
// partial sums from every rank's shared memory, 16 bytes a thread and all ranks' at once, and adds
// them in rank order.  (Sending them to that rank instead took 4 us more at 33 x 4096 x 14336.)
// X: void for tokens packed before; else their type, and the epilogue warps, idle until the last MMA,
// pack them: a warp a stage, 8 codes a lane, written in the order that TMA would have given.  Every
// CTA packs the K it needs.  Up to 8 tokens that is hidden behind the weights and saves a launch
// (4096 x 14336, MXFP4: 6.3 us against 8.9 for one token, 7.8 against 9.0 for 8, 11.2 against 9.5 for 12).
template <int FMT, int TOK, typename X>
__global__ void __launch_bounds__(kFewThreads, 2)
    block_gemm_few_kernel(const __grid_constant__ BlockGemmParams p, int split) {
  using C = FewCfg<FMT, TOK>;
  constexpr bool kPack = !std::is_void_v<X>;
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
  const int tokens = int(g.M);
  float* part = reinterpret_cast<float*>(smem);
  auto load_w = [&](int stage, int kb) {
    const uint32_t fb = smem_u32(&full[stage]);
    mbar_expect_tx(fb, kPack ? C::kW + C::kS : C::kStage);
    tma_load_2d(smW + stage * C::kW, &p.tmB, fb, kb * kRowBytes, tile * BM);
    tma_load_2d(smSW + stage * C::kS, &p.tmSB, fb, kb * C::G * 64, tile);
  };

  // The weights of the first stages are under way before anything else, and (b_ready) before the
  // kernel that packs the tokens is done.
  int early = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), kPack ? 2 : 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    mbar_init_fence();
    if (!g.b_ready) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (; early < nkb && early < STAGES; ++early) load_w(early, kb0 + early);
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), C::kCols);
  if constexpr (kPack) {  // rows that no token fills, and their scales, are zero in every stage
    if (warp >= 2) {
      for (int i = int(threadIdx.x) - 64; i < STAGES * C::kT / 16; i += 128)
        *reinterpret_cast<uint4*>(smem + STAGES * C::kW + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      for (int i = int(threadIdx.x) - 64; i < STAGES * C::kS / 16; i += 128)
        *reinterpret_cast<uint4*>(smem + STAGES * (C::kW + C::kT + C::kS) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float tensor_scale = 1.0f;  // of the tokens packed here
  __shared__ float factors[kPack && FMT == TE_NVFP4 ? kNvFactors : 1];
  if constexpr (kPack && FMT == TE_NVFP4) {
    tensor_scale = p.q.amax_in ? nv_scale_from_amax(*p.q.amax_in) : *p.q.scale;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      if (p.q.scale_out) *p.q.scale_out = tensor_scale;
      if (p.q.scale_inv_out) *p.q.scale_inv_out = __fdiv_rn(1.0f, tensor_scale);
    }
    nv_factors(factors, tensor_scale, int(threadIdx.x), kFewThreads);
    __syncthreads();
  }

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int i = 0; i < nkb; ++i) {
        if (!wait_or_abort(smem_u32(&empty[stage]), phase ^ 1, abort_flag, g.status)) break;
        if (i >= early) load_w(stage, kb0 + i);
        if constexpr (!kPack) {
          const uint32_t fb = smem_u32(&full[stage]);
          tma_load_2d(smT + stage * C::kT, &p.tmA, fb, (kb0 + i) * kRowBytes, 0);
          tma_load_2d(smST + stage * C::kS, &p.tmSA, fb, (kb0 + i) * C::G * 64, 0);
        }
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
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = block_idesc<FMT>(BM, TOK);
    const bool issuer = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nkb; ++i) {
      if (!warp_wait(smem_u32(&full[stage]), phase, abort_flag, g.status)) break;
      tc_fence_after();
      if (issuer) {
        stage_scales<FMT>(smSW + stage * C::kS, smST + stage * C::kS, tmem + C::kTsw, tmem + C::kTst);
        stage_mma<FMT, 1, 1>(tmem, smW + stage * C::kW, smT + stage * C::kT, tmem + C::kTsw, tmem + C::kTst, idesc,
                             i == 0);
        umma_commit<1>(smem_u32(&empty[stage]));
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (issuer) {
      umma_commit<1>(smem_u32(done));
      wait_bounded(smem_u32(done), 0, abort_flag, g.status, kDrainLimitNs, false);
    }
    __syncwarp();
  } else {
    if constexpr (kPack) {
      constexpr int kBlk = block_len(FMT);
      uint32_t amax = 0;
      bool ok = true;
      for (int i = warp - 2; i < nkb && ok; i += 4) {
        const int stage = i % STAGES;
        const int64_t col = int64_t(kb0 + i) * kStageK + lane * 8;
        const X* x = static_cast<const X*>(p.q.x) + col;
        uint8_t* codes = smem + STAGES * C::kW + stage * C::kT + (lane & 3) * 4;
        uint8_t* scales = smem + STAGES * (C::kW + C::kT + C::kS) + stage * C::kS;
        Eight<X> e[kFewPacked];
#pragma unroll
        for (int r = 0; r < int(kFewPacked); ++r) {
          if (col < g.K && r < tokens) e[r].load_fresh(x + r * g.K);
          else e[r].zero();
        }
        ok = warp_wait(smem_u32(&empty[stage]), ((i / STAGES) & 1) ^ 1, abort_flag, g.status);
        if (!ok) break;
#pragma unroll
        for (int r = 0; r < int(kFewPacked); ++r) {
          if (r >= tokens) break;
          uint32_t m = e[r].amax_bits();
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          if constexpr (kBlk == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
          amax = max(amax, m <= kInfBits ? m : 0u);
          const BlockScale b = block_scale<FMT>(m, tensor_scale, factors);
          float v[8];
          e[r].get(v);
          *reinterpret_cast<uint32_t*>(codes + r * kRowBytes + (((lane >> 2) ^ (r & 7)) << 4)) = codes8<FMT>(v, b).x;
          if (lane * 8 % kBlk == 0) scales[scale_offset(r, lane * 8 / kBlk)] = uint8_t(b.byte);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&full[stage]));
      }
      // every tile sees the same tokens: those of the first report the largest magnitude
      if (p.q.amax_out && tile == 0) {
        const float w = warp_max(__uint_as_float(amax));
        if (lane == 0) atomic_max_nonneg(p.q.amax_out, w);
      }
    }
    const int quad = warp & 3, row = quad * 32 + lane;
    const bool ok = warp_wait(smem_u32(done), 0, abort_flag, g.status);
    tc_fence_after();
    // the partial tile, [token][128 weight rows], over the pipeline's buffers: every stage has been
    // consumed (`done` follows the last MMA)
    const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16);
#pragma unroll 1
    for (int c = 0; c * 32 < tokens && ok; ++c) {
      uint32_t r[32];
      tmem_ld32(taddr + c * 32, r);
      tmem_ld_wait32(r);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c * 32 + i < tokens) part[(c * 32 + i) * BM + row] = __uint_as_float(r[i]);
    }
    tc_fence_before();
  }
  if (split > 1) cluster_sync();
  else __syncthreads();
  if (warp >= 2 && *abort_flag == 0) {
    // a warp on a token, 4 weight rows a thread
    float alpha = alpha_of(g);
    if constexpr (kPack && FMT == TE_NVFP4) alpha = __fdiv_rn(1.0f, tensor_scale) * alpha;
    const int64_t n = int64_t(tile) * BM + lane * 4;
    float b[4] = {};
    if (g.bias && n < g.N)
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = load_bias(g.bias, g.bias_dtype, n + i);
    for (int t = rank + (warp - 2) * split; t < tokens; t += 4 * split) {
      const uint32_t at = smem_u32(part + t * BM + lane * 4);
      float4 v[kMaxSplit];
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k)
        if (k < split) v[k] = ld_cluster4(map_to_rank(at, uint32_t(k)));
      float a[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int k = 1; k < kMaxSplit; ++k)
        if (k < split) {
          a[0] += v[k].x;
          a[1] += v[k].y;
          a[2] += v[k].z;
          a[3] += v[k].w;
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = fmaf(a[i], alpha, b[i]);
      store_four(g, t, n, a);
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();  // the partial tiles are read before any CTA of the cluster exits
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
bool code_map(CUtensorMap* tm, const void* ptr, int64_t rows, int64_t K, int64_t pitch, uint32_t box_rows) {
  return make_tmap_2d(tm, ptr, TE_E4M3, uint64_t(K / 2), uint64_t(rows), kRowBytes, box_rows, 128, uint64_t(pitch));
}

template <int FMT>
te_status launch_batch(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  using C = BatchCfg<FMT>;
  BlockGemmDev& g = prm.g;
  const uint64_t groups = uint64_t(scale_groups(FMT, a.K));
  g.num_m = int(ceil_div(a.M, BM * 2));
  g.num_n = int(ceil_div(a.N, BN));
  if (!code_map(&prm.tmA, a.A, a.M, a.K, 0, BM) || !code_map(&prm.tmB, a.B, a.N, a.K, a.b_pitch, C::kBRows) ||
      !make_tmap_scales(&prm.tmSA, a.a_scales, groups, uint64_t(ceil_div(a.M, 128)), C::G, 1) ||
      !make_tmap_scales(&prm.tmSB, a.b_scales, groups, uint64_t(ceil_div(a.N, 128)), C::G, 2) ||
      !make_tmap_2d(&prm.tmD, a.D, a.d_dtype, uint64_t(a.N), uint64_t(a.M), a.d_dtype == TE_F32 ? 16 : 32, 32, kOutRow))
    return TE_ERR_CUDA;
  const int64_t tile_bytes = int64_t(BM) * 2 * a.K / 2;
  const int64_t gm = (48ll << 20) / tile_bytes;  // A rows that a raster group may keep in L2
  g.group_m = int(gm < 4 ? 4 : gm < g.num_m ? gm : g.num_m);
  const int64_t tiles = int64_t(g.num_m) * g.num_n, slots = num_sms() / 2;
  if (tiles > 0x3fffffff) return TE_ERR_UNSUPPORTED;
  static PerDevice<bool> set;
  if (!allow_smem(block_gemm_kernel<FMT>, C::kSmem, set)) return TE_ERR_CUDA;
  return launch_clusters(block_gemm_kernel<FMT>, int(tiles < slots ? tiles : slots) * 2, kBatchThreads, C::kSmem,
                         2, s, prm, 0);
}

template <int FMT, int TOK, typename X>
te_status launch_few(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  using C = FewCfg<FMT, TOK>;
  const uint64_t groups = uint64_t(scale_groups(FMT, a.K));
  bool ok = code_map(&prm.tmB, a.B, a.N, a.K, a.b_pitch, BM) &&
            make_tmap_scales(&prm.tmSB, a.b_scales, groups, uint64_t(ceil_div(a.N, 128)), C::G, 1);
  if constexpr (std::is_void_v<X>)
    ok = ok && code_map(&prm.tmA, a.A, a.M, a.K, 0, TOK) && make_tmap_scales(&prm.tmSA, a.a_scales, groups, 1, C::G, 1);
  if (!ok) return TE_ERR_CUDA;
  const int64_t tiles = ceil_div(a.N, BM);
  if (tiles > 0x0fffffff) return TE_ERR_UNSUPPORTED;
  // K is split while all CTAs still fit on the device at once and each keeps two stages of K
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= 2 * num_sms() && split * 4 <= prm.g.num_kb) split *= 2;
  static PerDevice<bool> set;
  if (!allow_smem(block_gemm_few_kernel<FMT, TOK, X>, C::kSmem, set)) return TE_ERR_CUDA;
  return launch_clusters(block_gemm_few_kernel<FMT, TOK, X>, int(tiles) * split, kFewThreads, C::kSmem, split, s,
                         prm, split);
}

// The short side of the MMA that holds the tokens.
template <int FMT, typename X>
te_status launch_few_rows(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  static_assert(kFewPacked <= 16, "tokens packed in the kernel");
  if (!std::is_void_v<X> || a.M <= 16) return launch_few<FMT, 16, X>(a, prm, s);
  if constexpr (std::is_void_v<X>) {
    if (a.M <= 32) return launch_few<FMT, 32, X>(a, prm, s);
    if (a.M <= 48) return launch_few<FMT, 48, X>(a, prm, s);
    if (a.M <= 64) return launch_few<FMT, 64, X>(a, prm, s);
    return launch_few<FMT, 128, X>(a, prm, s);
  }
}

template <int FMT>
te_status launch_fmt(const BlockGemmArgs& a, BlockGemmParams& prm, cudaStream_t s) {
  // At 128 rows, few-row against batch kernel (MXFP4): 4096 x 14336 12.6 us against 20.3, 24576 x 8192 28.6
  // against 29.4, 28672 x 4096 19.7 against 16.9 (at 64 rows 15.7 against 16.5).
  return a.M <= 128 ? launch_few_rows<FMT, void>(a, prm, s) : launch_batch<FMT>(a, prm, s);
}

bool fill(const BlockGemmArgs& a, BlockGemmParams& prm) {
  memset(static_cast<void*>(&prm), 0, sizeof(prm));
  BlockGemmDev& g = prm.g;
  constexpr int64_t kMost = int64_t(1) << 30;  // tile coordinates are 32-bit, rounded up to whole tiles
  if (a.M > kMost || a.N > kMost || a.K > kMost) return false;
  g.M = a.M;
  g.N = a.N;
  g.K = a.K;
  g.num_kb = int(ceil_div(a.K, kStageK));
  g.a_scale_inv = a.a_scale_inv;
  g.b_scale_inv = a.b_scale_inv;
  g.bias = a.bias;
  g.bias_dtype = a.bias_dtype;
  g.D = a.D;
  g.d_dtype = a.d_dtype;
  g.b_ready = a.b_ready;
  g.status = device_status_ptr();
  return true;
}

}  // namespace

te_status launch_block_gemm(const BlockGemmArgs& a, cudaStream_t s) {
  if (a.M == 0 || a.N == 0) return TE_OK;
  BlockGemmParams prm;
  if (!fill(a, prm)) return TE_ERR_UNSUPPORTED;
  ProfileScope prof(TE_KERNEL_GEMM, s);
  return a.fmt == TE_NVFP4 ? launch_fmt<TE_NVFP4>(a, prm, s) : launch_fmt<TE_MXFP4>(a, prm, s);
}

te_status launch_block_gemm_packing(const BlockGemmArgs& a, const BlockQuantArgs& q, cudaStream_t s) {
  if (a.M == 0 || a.N == 0) return TE_OK;
  BlockGemmParams prm;
  if (a.M > kFewPacked || !fill(a, prm)) return TE_ERR_UNSUPPORTED;
  prm.q = q;
  ProfileScope prof(TE_KERNEL_GEMM, s);
  const bool f32 = q.x_dtype == TE_F32;
  if (a.fmt == TE_NVFP4)
    return f32 ? launch_few_rows<TE_NVFP4, float>(a, prm, s) : launch_few_rows<TE_NVFP4, __nv_bfloat16>(a, prm, s);
  return f32 ? launch_few_rows<TE_MXFP4, float>(a, prm, s) : launch_few_rows<TE_MXFP4, __nv_bfloat16>(a, prm, s);
}

}  // namespace te

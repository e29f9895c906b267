// What the residual norm's forward and backward kernels share: a thread's unit of 8 elements, parameter
// vectors asked for ahead of use, and the ring of rows in shared memory.
#pragma once

#include "cast.cuh"
#include "common.cuh"
#include "kernels.h"
#include "sync.cuh"

namespace te {

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Unit;

template <>
struct Unit<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* base, int64_t idx) {
    w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx);
  }
  __device__ __forceinline__ void load_const(const void* base, int64_t idx) {
    w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx));
  }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void cvt(f32x2 (&p)[4]) const {
    p[0] = bf16x2_f2(w.x);
    p[1] = bf16x2_f2(w.y);
    p[2] = bf16x2_f2(w.z);
    p[3] = bf16x2_f2(w.w);
  }
};

template <>
struct Unit<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t idx) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + idx);
    a = s[0];
    b = s[1];
  }
  __device__ __forceinline__ void load_const(const void* base, int64_t idx) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + idx);
    a = __ldg(s);
    b = __ldg(s + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void cvt(f32x2 (&p)[4]) const {
    p[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
    p[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
    p[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y));
    p[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
  }
};

template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t idx, const f32x2 (&p)[4]) {
  const float v[8] = {p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
  store_out<(sizeof(T) == 2 ? OUT_BF16 : OUT_F32), 8>(base, idx, v, CastState{});
}

// A unit of a parameter vector, as it lies in memory until it is used: asked for ahead of a barrier so
// that its way from L1 or L2 passes behind the barrier.
template <typename T>
struct Param {
  Unit<T> u;
  bool there;
  __device__ __forceinline__ void ask(const void* base, int64_t idx) {
    there = base != nullptr;
    if (there) u.load_const(base, idx);
  }
  // the values; `fill` without the vector
  __device__ __forceinline__ void get(f32x2 (&p)[4], float fill) const {
    if (there) {
      u.cvt(p);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2s(fill);
  }
};

__device__ __forceinline__ f32x2 sum8(const f32x2 (&v)[4]) { return add2(add2(v[0], v[1]), add2(v[2], v[3])); }

// ----------------------------------------------------------------------- the ring --------
// Shared memory of both kernels: "full" barriers, the abort flag, then `slots` slots of one row of
// each input.  The CTA's row k lies in slot k % slots; one thread refills the slot of row k - 1 after
// the first barrier of row k, which every thread passes with row k - 1 behind it.

constexpr int kMaxSlots = 3;
constexpr size_t kSmem = 227 * 1024;  // of one SM, shared by its CTAs
constexpr size_t kHeader = 128;

struct Ring {
  uint64_t* full;
  volatile int* abort_flag;
  uint8_t* data;
  uint32_t slot_bytes;
  int slots;
  int slot = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ Ring(uint8_t* smem, uint32_t bytes, int n)
      : full(reinterpret_cast<uint64_t*>(smem)),
        abort_flag(reinterpret_cast<volatile int*>(smem + kMaxSlots * 8)),
        data(smem + kHeader),
        slot_bytes(bytes),
        slots(n) {}
  __device__ __forceinline__ void init() {  // one thread; then a barrier
    for (int k = 0; k < slots; ++k) mbar_init(smem_u32(&full[k]), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  __device__ __forceinline__ const uint8_t* here() const { return data + uint32_t(slot) * slot_bytes; }
  // Whether the row in the current slot has arrived, to every lane of the warp.
  __device__ __forceinline__ bool wait(int* status) {
    const uint32_t bar = smem_u32(&full[slot]);
    int ok = 1;
    if ((threadIdx.x & 31) == 0 && !mbar_try_wait(bar, phase))
      ok = wait_bounded(bar, phase, abort_flag, status, kWaitLimitNs, true) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
  }
  __device__ __forceinline__ void next() {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ int before() const { return slot == 0 ? slots - 1 : slot - 1; }
  // After a failed wait: copies of rows k0 .. k1 - 1 land (or a short limit passes) before the CTA leaves.
  __device__ __forceinline__ void drain(int64_t k0, int64_t k1, int* status) {
    for (int64_t k = k0; k < k1; ++k)
      wait_bounded(smem_u32(&full[k % slots]), uint32_t(k / slots) & 1u, nullptr, status, kDrainLimitNs, false);
  }
};

// All threads of the CTA's G warps meet; whether `bad` was set in any.
template <int G>
__device__ __forceinline__ bool meet(bool bad) {
  if (G == 1) return __any_sync(0xffffffffu, bad);
  return __syncthreads_or(bad) != 0;
}

// CTAs of an SM (fewer than `ctas` where two slots of `bytes` would not fit each) and the slots of each, at
// most `most`: beyond what keeps the copies ahead, shared memory is better left to L1, which holds the
// parameter vectors.  (The carveout is left to the driver: all of it for shared memory cost the backward 8%.)
struct RingShape {
  int ctas, slots;
};
inline RingShape ring_shape(int ctas, size_t bytes, int most) {
  for (; ctas >= 1; ctas = ctas > 1 ? ctas / 2 : 0) {
    const size_t room = kSmem / ctas - 1024 - kHeader - 1536;  // 1 KB to the CTA itself, 1.5 KB static
    const size_t fit = room / bytes;
    if (fit >= 2) return RingShape{ctas, int(fit < size_t(most) ? fit : size_t(most))};
  }
  return RingShape{0, 0};
}

template <class K>
bool allow_smem(K kernel, PerDevice<bool>& done) {
  bool ok = false;
  return done.get(&ok, [&](bool* v) {
    *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem - 2048)) == cudaSuccess;
    return *v;
  });
}

}  // namespace te

// The global norm of many gradients and their clipping: n = sqrt(sum of g^2), out = g min(1, max / (n + eps)).
//
// The tensors go in a kernel's parameters, up to 512 of them a launch, so that a call needs no table
// in device memory and can be captured.  They are cut into chunks of 2048 vectors of 16 bytes; a CTA
// takes every grid-th chunk.  The squares pass is bound by reading; the scaling pass reads again (the
// last chunks first, which the squares pass left in L2) and writes.  353 MB: 68 + 102 us a call, with the
// results' way out of L2 in the next call's squares.  (Eight vectors to a thread, or the next chunk's
// asked for ahead, are no faster; two are 95 us for the 68.)
//
// Sums: a thread adds the squares of its 32 (bf16) or 16 (fp32) values of a chunk in fp32, and the
// chunks' sums, the warps' and the CTAs' as unevaluated pairs of fp32 (fp64 instructions are two orders slower
// here and would bound the small cases).  A square passes at most 11 roundings on its way into a pair (its
// chain's 8, one of an end of the tensor, two where the chains meet) and all terms are positive: the sum is
// within 11 * 2^-24, the norm within half of that and its own rounding, 2^-21.  Where a chunk's fp32 sum
// leaves [2^-80, 2^80] (a square overflowed, or small ones vanished), the thread takes that chunk's squares
// again in fp64, and so does every sum that they enter, so that this holds wherever the norm is a finite fp32.
#include "cast.cuh"
#include "common.cuh"
#include "kernels.h"

namespace te {

namespace {

constexpr int kThreads = 512;
constexpr int kVecs = 2048;              // vectors of 16 bytes in a chunk
constexpr int kPer = kVecs / kThreads;   // of a thread, all in flight at once
constexpr int kCtasPerSm = 3;
constexpr int kSmall = 32, kLarge = 512;  // tensors of one launch

template <int CAP>
struct Table {
  const void* src[CAP];
  void* dst[CAP];
  int64_t n[CAP];
  uint32_t first[CAP + 1];  // the tensor's first chunk
  uint8_t bf16[CAP];
  int count;
};

// A tensor cut at 16-byte boundaries of its source.
struct Cut {
  int64_t vecs;  // whole vectors
  int head;      // elements before them
  int tail;      // and behind
};

__host__ __device__ __forceinline__ Cut cut_of(const void* p, int64_t n, int es) {
  Cut c;
  const int64_t lead = int64_t((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es;
  c.head = int(lead < n ? lead : n);
  c.vecs = (n - c.head) / (16 / es);
  c.tail = int((n - c.head) % (16 / es));
  return c;
}

template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;  // the last tensor whose first chunk is at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float element(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_element(void* p, int64_t i, bool bf16, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

// hi + lo, the sum of some squares; lo the rounding errors of hi.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair add_pair(Pair a, Pair b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return Pair{s, (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo)};
}
__device__ __forceinline__ Pair warp_pair(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add_pair(v, Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

__device__ __forceinline__ double square64(const uint4& w, bool bf16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  double s = 0.0;
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const double lo = bf16_lo(u[i]), hi = bf16_hi(u[i]);
      s += lo * lo + hi * hi;
    } else {
      const double v = __uint_as_float(u[i]);
      s += v * v;
    }
  }
  return s;
}

// A thread's squares of a chunk (its vectors n, n + kThreads, ... read again) and of one end.
__device__ __noinline__ double chunk64(const uint4* v, int64_t n, int64_t vecs, float end, bool bf16) {
  double s = double(end) * double(end);
  for (int k = 0; k < kPer; ++k)
    if (n + k * kThreads < vecs) s += square64(v[n + k * kThreads], bf16);
  return s;
}

// Whether a value is not a zero (of either sign).
__device__ __forceinline__ bool nonzero(const uint4 (&w)[kPer], float end, bool bf16) {
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) any |= w[k].x | w[k].y | w[k].z | w[k].w;
  return (any & (bf16 ? 0x7fff7fffu : 0x7fffffffu)) != 0 || end != 0.0f;
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_squares_kernel(const __grid_constant__ Table<CAP> t,
                                                                                uint32_t chunks, GradSlot* slots) {
  __shared__ GradSlot red[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  Pair sum{0.0f, 0.0f};
  double rest = 0.0;  // squares taken in fp64
  // a thread's part of a chunk: its vectors, and one of the tensor's ends that no vector covers
  struct Part {
    const uint4* v;
    int64_t n, vecs;
    float end;
    bool bf16;
    uint4 w[kPer];
  };
  auto load = [&](uint32_t c, Part& q) {
    const int i = tensor_of(t, c);
    q.bf16 = t.bf16[i];
    const void* p = t.src[i];
    const Cut cut = cut_of(p, t.n[i], q.bf16 ? 2 : 4);
    const uint32_t at = c - t.first[i];
    q.v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + int64_t(cut.head) * (q.bf16 ? 2 : 4));
    q.n = int64_t(at) * kVecs + tid;
    q.vecs = cut.vecs;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      q.w[k] = q.n + k * kThreads < q.vecs ? q.v[q.n + k * kThreads] : make_uint4(0u, 0u, 0u, 0u);
    q.end = 0.0f;
    if (at == 0) {
      if (tid < cut.head) q.end = element(p, tid, q.bf16);
      else if (tid >= 32 && tid < 32 + cut.tail) q.end = element(p, t.n[i] - cut.tail + (tid - 32), q.bf16);
    }
  };
  auto add = [&](const Part& q) {
    f32x2 s0 = f2(q.end * q.end, 0.0f), s1 = f2s(0.0f);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (q.bf16) {
        f32x2 u[4];
        Pairs<__nv_bfloat16>::cvt(q.w[k], u);
        s0 = fma2(u[0], u[0], s0);
        s1 = fma2(u[1], u[1], s1);
        s0 = fma2(u[2], u[2], s0);
        s1 = fma2(u[3], u[3], s1);
      } else {
        f32x2 u[2];
        Pairs<float>::cvt(q.w[k], u);
        s0 = fma2(u[0], u[0], s0);
        s1 = fma2(u[1], u[1], s1);
      }
    }
    s0 = add2(s0, s1);
    const float s = f2lo(s0) + f2hi(s0);
    if (s >= 0x1p-80f && s <= 0x1p80f) sum = add_pair(sum, Pair{s, 0.0f});
    else if (nonzero(q.w, q.end, q.bf16)) rest += chunk64(q.v, q.n, q.vecs, q.end, q.bf16);
  };
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    Part q;
    load(c, q);
    add(q);
  }
  sum = warp_pair(sum);
  if (__any_sync(0xffffffffu, rest != 0.0)) rest = warp_sum64(rest);
  if ((tid & 31) == 0) red[tid >> 5] = GradSlot{sum.hi, sum.lo, rest};
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) {
      sum = add_pair(sum, Pair{red[w].hi, red[w].lo});
      if (red[w].rest != 0.0) rest += red[w].rest;
    }
    slots[blockIdx.x] = GradSlot{sum.hi, sum.lo, rest};
  }
}

// The norm from the slots, by one warp, in a fixed order: the same bits in every CTA, to every lane.
__device__ __forceinline__ double norm_of(const GradSlot* slots, int used, int lane) {
  Pair sum{0.0f, 0.0f};
  double rest = 0.0;
#pragma unroll 4
  for (int i = lane; i < used; i += 32) {
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(slots + i));
    sum = add_pair(sum, Pair{__uint_as_float(u.x), __uint_as_float(u.y)});
    if (u.z | u.w) rest += __hiloint2double(int(u.w), int(u.z));
  }
  sum = warp_pair(sum);
  double total = double(sum.hi) + double(sum.lo);
  if (__any_sync(0xffffffffu, rest != 0.0)) total += warp_sum64(rest);
  return sqrt(total);
}

__global__ void grad_norm_kernel(const GradSlot* slots, int used, float* norm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const double n = norm_of(slots, used, threadIdx.x);
  if (threadIdx.x == 0) *norm = float(n);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_clip_kernel(const __grid_constant__ Table<CAP> t,
                                                                             uint32_t chunks, const GradSlot* slots,
                                                                             int used, double max_norm, double eps,
                                                                             float* norm) {
  __shared__ float2 factor;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  if (tid < 32) {
    const double n = norm_of(slots, used, tid);
    if (tid == 0) {
      const double c = n + eps == 0.0 ? 1.0 : max_norm / (n + eps);
      // (a NaN stays one; a factor that fp32 holds in few bits or none is split into its power of two and the rest)
      if (c > 0.0 && c < 0x1p-100) {
        const int k = max(ilogb(c), -126);
        factor = make_float2(ldexpf(1.0f, k), float(ldexp(c, -k)));
      } else {
        factor = make_float2(1.0f, c > 1.0 ? 1.0f : float(c));
      }
      if (blockIdx.x == 0 && norm) *norm = float(n);
    }
  }
  __syncthreads();
  const float pre = factor.x, f = factor.y;
  const f32x2 pre2 = f2s(pre), f2v = f2s(f);
  // the last chunks first: they are what the squares pass has left in L2
  for (int64_t back = int64_t(chunks) - 1 - blockIdx.x; back >= 0; back -= gridDim.x) {
    const uint32_t c = uint32_t(back);
    const int i = tensor_of(t, c);
    const bool bf16 = t.bf16[i];
    const void* p = t.src[i];
    void* d = t.dst[i];
    if (f == 1.0f && p == d) continue;  // nothing changes
    const int es = bf16 ? 2 : 4;
    const Cut cut = cut_of(p, t.n[i], es);
    const uint32_t at = c - t.first[i];
    const int64_t n = t.n[i];
    const int64_t v0 = int64_t(at) * kVecs;
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(d)) & 15) == 0) {
      const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + int64_t(cut.head) * es);
      uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(d) + int64_t(cut.head) * es);
      uint4 w[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int64_t m = v0 + tid + k * kThreads;
        if (m < cut.vecs) w[k] = v[m];
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int64_t m = v0 + tid + k * kThreads;
        if (m >= cut.vecs) break;
        uint4 r;
        if (bf16) {
          f32x2 q[4];
          Pairs<__nv_bfloat16>::cvt(w[k], q);
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = mul2(mul2(q[e], pre2), f2v);
          r = make_uint4(pack_bf16x2(q[0].x, q[0].y), pack_bf16x2(q[1].x, q[1].y), pack_bf16x2(q[2].x, q[2].y),
                         pack_bf16x2(q[3].x, q[3].y));
        } else {
          f32x2 q[2];
          Pairs<float>::cvt(w[k], q);
          q[0] = mul2(mul2(q[0], pre2), f2v);
          q[1] = mul2(mul2(q[1], pre2), f2v);
          r = make_uint4(__float_as_uint(q[0].x), __float_as_uint(q[0].y), __float_as_uint(q[1].x),
                         __float_as_uint(q[1].y));
        }
        __stcs(o + m, r);
      }
    } else {  // ends of another alignment: one element at a time
      const int64_t e0 = cut.head + v0 * (16 / es);
      const int64_t last = v0 + kVecs < cut.vecs ? v0 + kVecs : cut.vecs;
      const int64_t e1 = cut.head + last * (16 / es);
      for (int64_t e = e0 + tid; e < e1; e += kThreads) store_element(d, e, bf16, element(p, e, bf16) * pre * f);
    }
    if (at == 0) {
      if (tid < cut.head) store_element(d, tid, bf16, element(p, tid, bf16) * pre * f);
      else if (tid >= 32 && tid < 32 + cut.tail) {
        const int64_t e = n - cut.tail + (tid - 32);
        store_element(d, e, bf16, element(p, e, bf16) * pre * f);
      }
    }
  }
}

int max_grid() { return num_sms() * kCtasPerSm; }

uint32_t chunks_of(const GradTensor& g) {
  const Cut c = cut_of(g.data, g.numel, g.dtype == TE_BF16 ? 2 : 4);
  const int64_t n = ceil_div(c.vecs, int64_t(kVecs));
  return uint32_t(n > 0 ? n : 1);
}

// Runs launch(table, chunks, grid) over the tensors, in batches of up to CAP.
template <int CAP, class Launch>
te_status batches(const GradTensor* g, int64_t count, Launch&& launch) {
  Table<CAP> t;
  for (int64_t i = 0; i < count;) {
    t.count = 0;
    uint64_t chunks = 0;
    for (; i < count && t.count < CAP; ++i) {
      if (g[i].numel == 0) continue;
      const uint64_t more = chunks_of(g[i]);
      if (chunks + more > 0x7fffffffull) {
        if (t.count == 0) return TE_ERR_UNSUPPORTED;
        break;
      }
      t.src[t.count] = g[i].data;
      t.dst[t.count] = g[i].out;
      t.n[t.count] = g[i].numel;
      t.bf16[t.count] = g[i].dtype == TE_BF16;
      t.first[t.count++] = uint32_t(chunks);
      chunks += more;
    }
    if (t.count == 0) break;
    t.first[t.count] = uint32_t(chunks);
    const int grid = int(chunks < uint64_t(max_grid()) ? chunks : uint64_t(max_grid()));
    const te_status st = launch(t, uint32_t(chunks), grid);
    if (st != TE_OK) return st;
  }
  return TE_OK;
}

template <int CAP>
te_status squares(const GradTensor* g, int64_t count, GradSlot* slots, int* used, cudaStream_t s) {
  return batches<CAP>(g, count, [&](const Table<CAP>& t, uint32_t chunks, int grid) {
    grad_squares_kernel<CAP><<<grid, kThreads, 0, s>>>(t, chunks, slots + *used);
    *used += grid;
    return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
  });
}

template <int CAP>
te_status clip(const GradTensor* g, int64_t count, const GradSlot* slots, int used, double max_norm, double eps,
               float* norm, cudaStream_t s) {
  return batches<CAP>(g, count, [&](const Table<CAP>& t, uint32_t chunks, int grid) {
    const te_status st = launch_dependent(grad_clip_kernel<CAP>, dim3(unsigned(grid)), dim3(kThreads), s, t, chunks,
                                          slots, used, max_norm, eps, norm);
    norm = nullptr;  // the first launch writes it
    return st;
  });
}

}  // namespace

size_t grad_norm_workspace(int64_t count) {
  if (count <= 0) return 0;
  return size_t(ceil_div(count, int64_t(kLarge)) + 1) * size_t(max_grid()) * sizeof(GradSlot);
}

te_status launch_grad_squares(const GradTensor* t, int64_t count, GradSlot* slots, int* used, cudaStream_t s) {
  ProfileScope prof(TE_KERNEL_QUANTIZE, s);
  *used = 0;
  return count <= kSmall ? squares<kSmall>(t, count, slots, used, s) : squares<kLarge>(t, count, slots, used, s);
}

te_status launch_grad_norm(const GradSlot* slots, int used, float* norm, cudaStream_t s) {
  ProfileScope prof(TE_KERNEL_QUANTIZE, s);
  return launch_dependent(grad_norm_kernel, dim3(1), dim3(32), s, slots, used, norm);
}

te_status launch_grad_clip(const GradTensor* t, int64_t count, const GradSlot* slots, int used, double max_norm,
                           double eps, float* norm, cudaStream_t s) {
  ProfileScope prof(TE_KERNEL_QUANTIZE, s);
  return count <= kSmall ? clip<kSmall>(t, count, slots, used, max_norm, eps, norm, s)
                         : clip<kLarge>(t, count, slots, used, max_norm, eps, norm, s);
}

}  // namespace te

// The norms around a residual stream (an addition of this library; the norm itself is that of the
// TransformerEngine JAX "LayerNorm MLP" page, Description, forward step (1)):
//   p = norm(y; post_gamma, post_beta) or y,  x_out = a * residual + gate * p,  out = norm(x_out)
// and its gradient.  Unfused this is four passes over rows in memory; here a row is read once,
// stays in registers, and its two results are written once.
//
// Both kernels give a row to a CTA, each thread holding NV units of 8 neighbouring elements.
#include "cast.cuh"
#include "common.cuh"
#include "kernels.h"

namespace te {

namespace {

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

// A parameter vector's unit, plus `shift` (one for a zero-centered gain); `fill` without the vector.
template <typename T>
__device__ __forceinline__ void param(const void* base, int64_t idx, float shift, float fill, f32x2 (&p)[4]) {
  if (base == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2s(fill);
    return;
  }
  Unit<T> u;
  u.load_const(base, idx);
  u.cvt(p);
  if (shift != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = add2(p[i], f2s(shift));
  }
}

// ----------------------------------------------------------------------- forward ---------

constexpr int kMaxWarps = 32;

// Mean and 1 / sqrt(variance + eps) of a row held by the CTA.  LayerNorm: each warp takes its own
// mean, then the squares about it, and the warps' (count, mean, squares) are joined about the row's
// mean, so that no sum of squares of a large mean is ever formed and one barrier serves both.
template <bool LN, int NV>
__device__ __forceinline__ float2 row_stats(const f32x2 (&v)[NV][4], int first, int threads, int units, float inv_h,
                                            float eps, float2* red, const float* counts) {
  const int lane = first & 31, warp = first >> 5, warps = threads >> 5;
  float mean_w = 0.0f;
  if (LN) {
    f32x2 s = f2s(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (first + i * threads < units) s = add2(s, add2(add2(v[i][0], v[i][1]), add2(v[i][2], v[i][3])));
    }
    const float n = counts[warp];
    mean_w = n > 0.0f ? warp_sum(f2lo(s) + f2hi(s)) / n : 0.0f;
  }
  const f32x2 m2 = f2s(mean_w);
  f32x2 q = f2s(0.0f), q1 = f2s(0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (first + i * threads < units) {
#pragma unroll
      for (int p = 0; p < 4; p += 2) {
        const f32x2 d0 = LN ? sub2(v[i][p], m2) : v[i][p], d1 = LN ? sub2(v[i][p + 1], m2) : v[i][p + 1];
        q = fma2(d0, d0, q);
        q1 = fma2(d1, d1, q1);
      }
    }
  }
  q = add2(q, q1);
  const float sq = warp_sum(f2lo(q) + f2hi(q));
  if (lane == 0) red[warp] = make_float2(mean_w, sq);
  __syncthreads();
  float mean = 0.0f, var = 0.0f;
  if (LN) {
    for (int w = 0; w < warps; ++w) mean += counts[w] * red[w].x;
    mean *= inv_h;
  }
  for (int w = 0; w < warps; ++w) {
    const float2 r = red[w];
    const float d = r.x - mean;
    var += LN ? r.y + counts[w] * (d * d) : r.y;
  }
  return make_float2(mean, rsqrtf(var * inv_h + eps));
}

template <typename TY, typename TR, bool LN, bool POST, int NV, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) residual_norm_fwd_kernel(ResidualNormArgs a) {
  // the kernel after this one may launch its setup now (it waits for this grid's completion)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float2 red[4][kMaxWarps];
  __shared__ float counts[kMaxWarps];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int units = int(a.H / 8);
  if (tid < kMaxWarps) {  // elements that warp `tid` holds
    int n = 0;
    for (int i = 0; i < NV; ++i) n += max(0, min(32, units - (tid * 32 + i * threads)));
    counts[tid] = float(8 * n);
  }
  __syncthreads();
  const CastState cs = cast_begin(a.cast);
  const int kind = out_kind(cs);
  const bool want_amax = a.cast.amax_out != nullptr;
  const float inv_h = 1.0f / float(a.H);
  const float shift = a.zero_centered_gamma ? 1.0f : 0.0f;
  const f32x2 scale2 = f2s(a.residual_scale);
  float amax = 0.0f;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, par ^= 1) {
    const int64_t base = row * a.H;
    Unit<TY> y[NV];
    Unit<TR> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = tid + i * threads;
      if (u < units) {
        y[i].load(a.y, base + int64_t(u) * 8);
        r[i].load(a.residual, base + int64_t(u) * 8);
      } else {
        y[i].zero();
        r[i].zero();
      }
    }
    f32x2 x[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i].cvt(x[i]);
    if (POST) {
      const float2 st = row_stats<LN, NV>(x, tid, threads, units, inv_h, a.eps, red[2 + par], counts);
      if (tid == 0) {
        if (a.post_mu) a.post_mu[row] = st.x;
        if (a.post_rsigma) a.post_rsigma[row] = st.y;
      }
      const f32x2 mean2 = f2s(st.x), rs2 = f2s(st.y);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int u = tid + i * threads;
        if (u < units) {
          f32x2 g[4], b[4];
          param<TY>(a.post_gamma, int64_t(u) * 8, shift, 1.0f, g);
          if (LN) param<TY>(a.post_beta, int64_t(u) * 8, 0.0f, 0.0f, b);
#pragma unroll
          for (int p = 0; p < 4; ++p)
            x[i][p] = LN ? fma2(sub2(x[i][p], mean2), mul2(g[p], rs2), b[p]) : mul2(mul2(x[i][p], rs2), g[p]);
        }
      }
    }
    const int64_t gate_at = a.gate ? row / a.gate_rows * a.H : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = tid + i * threads;
      if (u < units) {
        f32x2 rp[4];
        r[i].cvt(rp);
        if (a.gate) {
          f32x2 g[4];
          param<TY>(a.gate, gate_at + int64_t(u) * 8, 0.0f, 1.0f, g);
#pragma unroll
          for (int p = 0; p < 4; ++p) x[i][p] = mul2(x[i][p], g[p]);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) x[i][p] = fma2(scale2, rp[p], x[i][p]);
        if (kind != OUT_NONE) store8<TR>(a.x_out, base + int64_t(u) * 8, x[i]);
      }
    }
    const float2 st = row_stats<LN, NV>(x, tid, threads, units, inv_h, a.eps, red[par], counts);
    if (tid == 0) {
      if (a.mu) a.mu[row] = st.x;
      if (a.rsigma) a.rsigma[row] = st.y;
    }
    const f32x2 mean2 = f2s(st.x), rs2 = f2s(st.y);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = tid + i * threads;
      if (u < units) {
        f32x2 g[4], b[4];
        param<TY>(a.gamma, int64_t(u) * 8, shift, 1.0f, g);
        if (LN) param<TY>(a.beta, int64_t(u) * 8, 0.0f, 0.0f, b);
        float o[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const f32x2 v = LN ? fma2(sub2(x[i][p], mean2), mul2(g[p], rs2), b[p]) : mul2(mul2(x[i][p], rs2), g[p]);
          if (want_amax) amax = absmax2(amax, v);
          o[2 * p] = f2lo(v);
          o[2 * p + 1] = f2hi(v);
        }
        const int64_t at = base + int64_t(u) * 8;
        switch (kind) {
          case OUT_F32: store_out<OUT_F32, 8>(a.out, at, o, cs); break;
          case OUT_BF16: store_out<OUT_BF16, 8>(a.out, at, o, cs); break;
          case OUT_E4M3: store_out<OUT_E4M3, 8>(a.out, at, o, cs); break;
          default: break;
        }
      }
    }
  }
  if (want_amax) {
    amax = warp_max(amax);
    if ((tid & 31) == 0) atomic_max_nonneg(a.cast.amax_out, amax);
  }
}

template <typename TY, typename TR, bool LN, bool POST, int NV, int THREADS, int CTAS>
te_status fwd_launch(const ResidualNormArgs& a, int threads, cudaStream_t s) {
  const int64_t n = int64_t(num_sms()) * (threads <= 128 ? 8 : threads <= 256 ? 4 : 2);
  const unsigned grid = unsigned(a.M < n ? a.M : n);
  residual_norm_fwd_kernel<TY, TR, LN, POST, NV, THREADS, CTAS><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

inline int round_warp(int64_t n) { return int((n + 31) / 32 * 32); }

template <typename TY, typename TR, bool LN, bool POST>
te_status fwd_shape(const ResidualNormArgs& a, cudaStream_t s) {
  const int64_t units = a.H / 8;
  if (units <= 128 || a.M <= num_sms()) return fwd_launch<TY, TR, LN, POST, 1, 1024, 1>(a, round_warp(units), s);
  if (units <= 256) return fwd_launch<TY, TR, LN, POST, 2, 256, 2>(a, round_warp((units + 1) / 2), s);
  return fwd_launch<TY, TR, LN, POST, 4, 256, 2>(a, round_warp((units + 3) / 4), s);
}

// ----------------------------------------------------------------------- backward --------

// Sums of two values over the CTA, the warps' added in warp order (the same bits in every thread).
__device__ __forceinline__ float2 row_sums(float a, float b, int tid, int threads, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((tid & 31) == 0) red[tid >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = red[0];
  for (int w = 1; w < (threads >> 5); ++w) {
    t.x += red[w].x;
    t.y += red[w].y;
  }
  return t;
}

constexpr int kBwdNV = 2;
constexpr int kBwdThreads = 512;

// A CTA takes neighbouring rows.  With S1 = the sum of dx * phat and S2 = that of dx over the rows
// that share a gate (phat the normalized y, or y itself without a post norm), the gradients of the
// gate and of the post norm's gain and shift are
//   dgate = post_g * S1 + post_b * S2,  dpost_gamma = sum over gates of gate * S1,
//   dpost_beta = sum over gates of gate * S2,
// so a thread keeps two sums for these three.  They are written where a gate's rows end: the part of
// CTA c's rows that gate row g serves is slot c + g, which no other part has (c or g grows from one
// part to the next).
template <typename TY, typename TR, bool LN, bool POST, bool SUMS>
__global__ void __launch_bounds__(kBwdThreads, 1) residual_norm_bwd_kernel(ResidualNormBwdArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int NV = kBwdNV;
  __shared__ float2 red[4][kBwdThreads / 32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int units = int(a.H / 8);
  const float inv_h = 1.0f / float(a.H);
  const float shift = a.zero_centered_gamma ? 1.0f : 0.0f;
  f32x2 ag[NV][4], ab[NV][4], s1[NV][4], s2[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int p = 0; p < 4; ++p) ag[i][p] = ab[i][p] = s1[i][p] = s2[i][p] = f2s(0.0f);
  const int64_t r0 = int64_t(blockIdx.x) * a.rows_per_cta;
  const int64_t r1 = r0 + a.rows_per_cta < a.M ? r0 + a.rows_per_cta : a.M;
  int64_t gate_row = r0 / a.gate_rows;
  int64_t gate_end = (gate_row + 1) * a.gate_rows;
  // column sums [2][H] of this thread's units
  auto write = [&](float* dst, const f32x2 (&u)[NV][4], const f32x2 (&v)[NV][4], bool second) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = tid + i * threads;
      if (n < units) {
        store8<float>(dst, int64_t(n) * 8, u[i]);
        if (second) store8<float>(dst + a.H, int64_t(n) * 8, v[i]);
      }
    }
  };
  int par = 0;
  for (int64_t row = r0; row < r1; ++row, par ^= 1) {
    const int64_t base = row * a.H;
    const float mu = LN ? a.mu[row] : 0.0f, rs = a.rsigma[row];
    Unit<TY> dout[NV], y[NV];
    Unit<TR> x[NV], dxo[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = base + int64_t(tid + i * threads) * 8;
      dout[i].zero();
      x[i].zero();
      dxo[i].zero();
      y[i].zero();
      if (tid + i * threads < units) {
        dout[i].load(a.dout, at);
        x[i].load(a.x_out, at);
        if (a.dx_out) dxo[i].load(a.dx_out, at);
        if (SUMS) y[i].load(a.y, at);
      }
    }
    f32x2 xh[NV][4], dx[NV][4];  // xhat; dout * g, then dx
    f32x2 t1 = f2s(0.0f), t2 = f2s(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = tid + i * threads;
#pragma unroll
      for (int p = 0; p < 4; ++p) xh[i][p] = dx[i][p] = f2s(0.0f);
      if (u < units) {
        f32x2 g[4], d[4], xp[4];
        param<TY>(a.gamma, int64_t(u) * 8, shift, 1.0f, g);
        dout[i].cvt(d);
        x[i].cvt(xp);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          xh[i][p] = LN ? mul2(sub2(xp[p], f2s(mu)), f2s(rs)) : mul2(xp[p], f2s(rs));
          dx[i][p] = mul2(d[p], g[p]);
          if (LN) t1 = add2(t1, dx[i][p]);
          t2 = fma2(dx[i][p], xh[i][p], t2);
          ag[i][p] = fma2(d[p], xh[i][p], ag[i][p]);
          if (LN) ab[i][p] = add2(ab[i][p], d[p]);
        }
      }
    }
    const float2 m = row_sums(f2lo(t1) + f2hi(t1), f2lo(t2) + f2hi(t2), tid, threads, red[par]);
    const f32x2 c1 = f2s(-rs * (m.x * inv_h)), c2 = f2s(-rs * (m.y * inv_h)), rs2 = f2s(rs);
    const int64_t gate_at = gate_row * a.H;
    const float pmu = POST && LN ? a.post_mu[row] : 0.0f, prs = POST ? a.post_rsigma[row] : 0.0f;
    t1 = t2 = f2s(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = tid + i * threads;
      if (u < units) {
        const int64_t at = base + int64_t(u) * 8;
        f32x2 d[4];
        dxo[i].cvt(d);
#pragma unroll
        for (int p = 0; p < 4; ++p)
          dx[i][p] = add2(d[p], fma2(xh[i][p], c2, LN ? fma2(dx[i][p], rs2, c1) : mul2(dx[i][p], rs2)));
        if (a.dresidual) {
          f32x2 o[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) o[p] = mul2(dx[i][p], f2s(a.residual_scale));
          store8<TR>(a.dresidual, at, o);
        }
        if (SUMS) {
          f32x2 gt[4];
          param<TY>(a.gate, gate_at + int64_t(u) * 8, 0.0f, 1.0f, gt);
          y[i].cvt(xh[i]);  // phat from here on
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            if (POST) xh[i][p] = LN ? mul2(sub2(xh[i][p], f2s(pmu)), f2s(prs)) : mul2(xh[i][p], f2s(prs));
            s1[i][p] = fma2(dx[i][p], xh[i][p], s1[i][p]);
            if (POST && LN) s2[i][p] = add2(s2[i][p], dx[i][p]);
            dx[i][p] = mul2(dx[i][p], gt[p]);
          }
        }
        if (POST) {
          f32x2 g[4];
          param<TY>(a.post_gamma, int64_t(u) * 8, shift, 1.0f, g);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            dx[i][p] = mul2(dx[i][p], g[p]);
            if (LN) t1 = add2(t1, dx[i][p]);
            t2 = fma2(dx[i][p], xh[i][p], t2);
          }
        } else if (a.dy) {
          store8<TY>(a.dy, at, dx[i]);
        }
      }
    }
    if (POST) {
      const float2 n = row_sums(f2lo(t1) + f2hi(t1), f2lo(t2) + f2hi(t2), tid, threads, red[2 + par]);
      const f32x2 d1 = f2s(-prs * (n.x * inv_h)), d2 = f2s(-prs * (n.y * inv_h)), p2 = f2s(prs);
      if (a.dy) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int u = tid + i * threads;
          if (u < units) {
            f32x2 o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
              o[p] = fma2(xh[i][p], d2, LN ? fma2(dx[i][p], p2, d1) : mul2(dx[i][p], p2));
            store8<TY>(a.dy, base + int64_t(u) * 8, o);
          }
        }
      }
    }
    if (SUMS && (row + 1 == gate_end || row + 1 == r1)) {
      write(a.gate_partials + (int64_t(blockIdx.x) + gate_row) * 2 * a.H, s1, s2, POST && LN);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) s1[i][p] = s2[i][p] = f2s(0.0f);
      ++gate_row;
      gate_end += a.gate_rows;
    }
  }
  write(a.partials + int64_t(blockIdx.x) * 2 * a.H, ag, ab, LN);
}

// The columns' sums over the CTAs (and, of S1 and S2, over the parts of each gate's rows), in a fixed
// order.  A CTA takes 128 columns, four to a lane; its warps take the terms w, w + 16, ... and are
// added in warp order.
constexpr int kSumWarps = 16;

struct Sum2 {
  float4 a, b;
};
__device__ __forceinline__ void add4(float4& t, const float4& v) {
  t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
}
__device__ __forceinline__ void fma4(float4& t, const float4& u, const float4& v) {
  t.x = fmaf(u.x, v.x, t.x); t.y = fmaf(u.y, v.y, t.y); t.z = fmaf(u.z, v.z, t.z); t.w = fmaf(u.w, v.w, t.w);
}

template <typename TY>
__device__ __forceinline__ float4 param4(const void* base, int64_t j, float shift, float fill) {
  if (base == nullptr) return make_float4(fill, fill, fill, fill);
  if (sizeof(TY) == 2) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + j));
    return make_float4(bf16_lo(w.x) + shift, bf16_hi(w.x) + shift, bf16_lo(w.y) + shift, bf16_hi(w.y) + shift);
  }
  const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + j));
  return make_float4(v.x + shift, v.y + shift, v.z + shift, v.w + shift);
}

// The warps' terms of one column block joined in warp order; the result is in warp 0.
__device__ __forceinline__ Sum2 join(Sum2 v, Sum2 (*box)[32], int w, int lane) {
  box[w][lane] = v;
  __syncthreads();
  if (w == 0) {
    for (int k = 1; k < kSumWarps; ++k) {
      add4(v.a, box[k][lane].a);
      add4(v.b, box[k][lane].b);
    }
  }
  __syncthreads();
  return v;
}

template <typename TY>
__global__ void __launch_bounds__(kSumWarps * 32) residual_norm_bwd_sum_kernel(ResidualNormBwdArgs a, int ctas,
                                                                               bool second) {
  __shared__ Sum2 box[kSumWarps][32];
  // launched as a programmatic dependent of the kernel that writes the partials
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t j = int64_t(blockIdx.x) * 128 + lane * 4;  // H is a multiple of 8
  const bool in = j < a.H;
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto at = [&](const float* p) { return *reinterpret_cast<const float4*>(p); };
  if (blockIdx.y == 0) {
    Sum2 t{zero, zero};
    if (in) {
#pragma unroll 4
      for (int c = w; c < ctas; c += kSumWarps) {
        const float* p = a.partials + int64_t(c) * 2 * a.H + j;
        add4(t.a, at(p));
        if (second) add4(t.b, at(p + a.H));
      }
    }
    t = join(t, box, w, lane);
    if (w == 0 && in) {
      a.dgamma[j] = t.a.x; a.dgamma[j + 1] = t.a.y; a.dgamma[j + 2] = t.a.z; a.dgamma[j + 3] = t.a.w;
      if (second && a.dbeta) {
        a.dbeta[j] = t.b.x; a.dbeta[j + 1] = t.b.y; a.dbeta[j + 2] = t.b.z; a.dbeta[j + 3] = t.b.w;
      }
    }
    return;
  }
  const bool post = a.post_gamma != nullptr, two = post && second;
  const float shift = a.zero_centered_gamma ? 1.0f : 0.0f;
  const float4 g1 = in && post ? param4<TY>(a.post_gamma, j, shift, 1.0f) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  const float4 b1 = in && two ? param4<TY>(a.post_beta, j, 0.0f, 0.0f) : zero;
  const int64_t gates = a.M / a.gate_rows;
  // S1 and S2 of gate row g: the slots c + g of the CTAs c that hold its rows, every `step`-th
  auto gate_sums = [&](int64_t g, int64_t from, int64_t step) {
    Sum2 t{zero, zero};
    const int64_t c0 = g * a.gate_rows / a.rows_per_cta, c1 = ((g + 1) * a.gate_rows - 1) / a.rows_per_cta;
#pragma unroll 4
    for (int64_t c = c0 + from; c <= c1; c += step) {
      const float* p = a.gate_partials + (c + g) * 2 * a.H + j;
      add4(t.a, at(p));
      if (two) add4(t.b, at(p + a.H));
    }
    return t;
  };
  Sum2 dp{zero, zero};
  auto finish = [&](int64_t g, const Sum2& s) {
    if (a.dgate) {
      float4 o = zero;
      fma4(o, g1, s.a);
      if (two) fma4(o, b1, s.b);
      float* d = a.dgate + g * a.H + j;
      d[0] = o.x; d[1] = o.y; d[2] = o.z; d[3] = o.w;
    }
    const float4 gt = param4<TY>(a.gate, g * a.H + j, 0.0f, 1.0f);
    fma4(dp.a, gt, s.a);
    if (two) fma4(dp.b, gt, s.b);
  };
  if (gates < kSumWarps) {  // few gates: the warps share the parts of each
    for (int64_t g = 0; g < gates; ++g) {
      Sum2 t{zero, zero};
      if (in) t = gate_sums(g, w, kSumWarps);
      t = join(t, box, w, lane);
      if (w == 0 && in) finish(g, t);
    }
  } else {  // many: each warp takes whole gates
    if (in)
      for (int64_t g = w; g < gates; g += kSumWarps) finish(g, gate_sums(g, 0, 1));
    dp = join(dp, box, w, lane);
  }
  if (w == 0 && in && post) {
    if (a.dpost_gamma) {
      float* d = a.dpost_gamma + j;
      d[0] = dp.a.x; d[1] = dp.a.y; d[2] = dp.a.z; d[3] = dp.a.w;
    }
    if (two && a.dpost_beta) {
      float* d = a.dpost_beta + j;
      d[0] = dp.b.x; d[1] = dp.b.y; d[2] = dp.b.z; d[3] = dp.b.w;
    }
  }
}

struct BwdShape {
  int threads;
  int64_t ctas, rows_per_cta;
};
// 16 warps to an SM, in as many CTAs as the row's width leaves room for.
BwdShape bwd_shape(int64_t M, int64_t H) {
  BwdShape s;
  s.threads = round_warp((H / 8 + kBwdNV - 1) / kBwdNV);
  const int64_t n = int64_t(num_sms()) * (kBwdThreads / s.threads);
  s.rows_per_cta = M > n ? ceil_div(M, n) : 1;
  s.ctas = ceil_div(M, s.rows_per_cta);
  return s;
}

template <typename TY, typename TR, bool LN, bool POST, bool SUMS>
te_status bwd_launch(ResidualNormBwdArgs a, cudaStream_t s) {
  const BwdShape sh = bwd_shape(a.M, a.H);
  a.rows_per_cta = sh.rows_per_cta;
  a.gate_partials = a.partials + sh.ctas * 2 * a.H;
  residual_norm_bwd_kernel<TY, TR, LN, POST, SUMS><<<unsigned(sh.ctas), sh.threads, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return TE_ERR_CUDA;
  return launch_dependent(residual_norm_bwd_sum_kernel<TY>, dim3(unsigned(ceil_div(a.H, 128)), SUMS ? 2 : 1),
                          dim3(kSumWarps * 32), s, a, int(sh.ctas), LN);
}

template <typename TY, typename TR>
te_status fwd_types(const ResidualNormArgs& a, cudaStream_t s) {
  const bool post = a.post_gamma != nullptr;
  if (a.norm_type == TE_LAYERNORM)
    return post ? fwd_shape<TY, TR, true, true>(a, s) : fwd_shape<TY, TR, true, false>(a, s);
  return post ? fwd_shape<TY, TR, false, true>(a, s) : fwd_shape<TY, TR, false, false>(a, s);
}

template <typename TY, typename TR, bool LN>
te_status bwd_norm(const ResidualNormBwdArgs& a, cudaStream_t s) {
  if (a.post_gamma) return bwd_launch<TY, TR, LN, true, true>(a, s);
  return a.gate ? bwd_launch<TY, TR, LN, false, true>(a, s) : bwd_launch<TY, TR, LN, false, false>(a, s);
}

template <typename TY, typename TR>
te_status bwd_types(const ResidualNormBwdArgs& a, cudaStream_t s) {
  return a.norm_type == TE_LAYERNORM ? bwd_norm<TY, TR, true>(a, s) : bwd_norm<TY, TR, false>(a, s);
}

}  // namespace

te_status launch_residual_norm_fwd(const ResidualNormArgs& a, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_NORM_FWD, s);
  if (a.y_dtype == TE_F32) return fwd_types<float, float>(a, s);
  return a.residual_dtype == TE_F32 ? fwd_types<__nv_bfloat16, float>(a, s)
                                    : fwd_types<__nv_bfloat16, __nv_bfloat16>(a, s);
}

size_t residual_norm_bwd_workspace(int64_t M, int64_t H, int64_t gates) {
  if (M <= 0 || H <= 0) return 0;
  const int64_t slots = bwd_shape(M, H).ctas + (gates > 0 ? gates : 1);
  return size_t(bwd_shape(M, H).ctas + slots) * 2 * size_t(H) * sizeof(float);
}

te_status launch_residual_norm_bwd(const ResidualNormBwdArgs& a, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_NORM_BWD, s);
  if (a.dtype == TE_F32) return bwd_types<float, float>(a, s);
  return a.residual_dtype == TE_F32 ? bwd_types<__nv_bfloat16, float>(a, s)
                                    : bwd_types<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace te

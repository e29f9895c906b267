// Activation gradient + bias gradient (+ E4M3 cast) from an 8-bit checkpoint of the activation's
// input, with the activation itself recomputed in the same pass.
//
// The forward keeps h in MXFP8 (E4M3 codes, one power-of-two scale for 32 neighbours) instead of
// bf16.  The backward needs act'(h) for the gradient and act(h) as an operand of the second
// kernel's gradient; both share one logistic (or exponential) of the h that was just decoded:
//   dx = dy * act'(h),  a = act(h);   gated: [dy * l * act'(g) | dy * act(g)],  a = act(g) * l.
// Decoding is exact in fp32 (4 significant bits times a power of two).
//
// Bound by memory: with bf16 dy, dx and a, 2 + 1.03 + 2 + 2 bytes an element; 16384 x 16384 gelu takes
// 301 us (92% of the copy rate), relu 290 (96%), 8192 x 14336 swiglu 191 us (91%), geglu 192, with E4M3 dx
// 163 (86%).  Current scaling takes two passes, the first for the amax, each reading dy and codes and
// computing the derivative: 258 us.  In fp32 8192 x 16384 silu takes 293 us (88%), gelu 295, but 8192 x
// 14336 swiglu 457 (69%) and geglu 449: three CTAs an SM leave 80 registers, and the fp32 gated forms
// spill 940 to 1020 bytes a thread, the bf16 gated ones 310 to 440, gelu in bf16 16, fp32 plain 16 to 230
// (bf16 relu and silu none).  Two CTAs an SM spill nothing: fp32 swiglu 378 us, but bf16 198 and with E4M3
// dx 177.  A CTA owns a strip
// of 256 columns (8 a lane: 16 bytes of dy, 8 of codes) and 128 rows, the rows of one row of
// scale tiles; the strip's scales are decoded to fp32 in shared memory once.  The column sums go
// the way of dact_dbias_kernel: registers, warps in order, one partial row a CTA, and an ordered
// sum of the partial rows, so dbias is the same on every run.
#include "block.cuh"
#include "cast.cuh"

namespace te {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 128;  // rows of a CTA = of a scale tile = of a dbias partial
constexpr int kCols = 256;
constexpr int kSb = kCols / 32;

// Inputs are read by ordinary loads, not through the read-only path: this grid may be running while the
// kernel before it still writes them.  Written out, since nothing that this kernel stores is read by them:
// the compiler's own loads stay ahead of the stores, which costs registers (8192 x 14336 swiglu 199 us
// against 191).  Their addresses depend on a value made behind the wait.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <typename T>
struct Dy8;
template <>
struct Dy8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    u = load16(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const { Pairs<__nv_bfloat16>::cvt(u, v); }
};
template <>
struct Dy8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = load16(static_cast<const float*>(p) + i);
    b = load16(static_cast<const float*>(p) + i + 4);
  }
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const {
    v[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
    v[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y));
    v[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
  }
};

__device__ __forceinline__ void decode8(const uint2& c, float f, f32x2 (&h)[4]) {
  const f32x2 s = f2s(f);
  h[0] = mul2(unpack_e4m3x2(uint16_t(c.x)), s);
  h[1] = mul2(unpack_e4m3x2(uint16_t(c.x >> 16)), s);
  h[2] = mul2(unpack_e4m3x2(uint16_t(c.y)), s);
  h[3] = mul2(unpack_e4m3x2(uint16_t(c.y >> 16)), s);
}

// exp2 arguments stop here: 1 / (1 + 2^126.5) flushes to zero, so that the logistic of a very
// negative argument is exactly zero (and e * s with it) and no product with it can overflow.
constexpr float kExp2Top = 126.5f;

// max and min that hand a NaN on, where fmaxf and fminf drop it.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// act(h) and act'(h) from one exponential and one reciprocal.  Both are NaN where h is: the format keeps
// an infinity as a NaN block, and 32 zero gradients in its place would hide it.  (Here ReLU does so too,
// unlike the kernels that read h itself, where a NaN counts as not positive.)
template <int ACT>
__device__ __forceinline__ void act_both(f32x2 h, f32x2& y, f32x2& d) {
  if constexpr (ACT == TE_RELU) {
    y = f2(max_nan(f2lo(h), 0.0f), max_nan(f2hi(h), 0.0f));
    d = f2(f2lo(h) > 0.0f ? 1.0f : f2lo(y), f2hi(h) > 0.0f ? 1.0f : f2hi(y));  // y: 0 or NaN there
  } else if constexpr (ACT == TE_SILU) {
    const f32x2 e = ex2_2(min2s(mul2(h, f2s(-kLog2e)), kExp2Top));
    const f32x2 s = rcp2(add2(e, f2s(1.0f)));
    y = mul2(h, s);
    d = mul2(s, fma2(h, mul2(e, s), f2s(1.0f)));
  } else {
    // beyond +-100 the logistic is 0 or 1 in fp32; the cube must not overflow
    const f32x2 c = f2(min_nan(max_nan(f2lo(h), -100.0f), 100.0f), min_nan(max_nan(f2hi(h), -100.0f), 100.0f));
    const f32x2 cc = mul2(c, c);
    const f32x2 e = ex2_2(min2s(mul2(c, fma2(cc, f2s(kGeluA2), f2s(kGeluA1))), kExp2Top));
    const f32x2 s = rcp2(add2(e, f2s(1.0f)));
    const f32x2 q = mul2(c, fma2(cc, f2s(6.0f * kGeluK0 * kGeluK1), f2s(2.0f * kGeluK0)));
    y = mul2(h, s);
    d = fma2(q, mul2(s, mul2(e, s)), s);
  }
}

__device__ __forceinline__ void flat8(const f32x2 (&p)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = f2lo(p[i]);
    v[2 * i + 1] = f2hi(p[i]);
  }
}

// (Fewer rows a CTA, for more CTAs where there are few, cost more in first loads than the tail gains:
// 777 x 14336 swiglu 31 us with 32 rows against 26.)
template <typename T, int ACT>
__global__ void __launch_bounds__(kWarps * 32, 3) dact_ckpt_kernel(DactCkptArgs a) {
  constexpr bool kGated = is_gated(ACT);
  constexpr int kBase = gate_act(ACT);
  constexpr int U = 2;  // rows that a warp loads together, twice that in flight
  constexpr int kPlain = sizeof(T) == 4 ? OUT_F32 : OUT_BF16;
  __shared__ float sc[kGated ? 2 : 1][kRows][kSb];
  __shared__ float red[kWarps][kGated ? 2 : 1][kCols];
  // the column-sum kernel that follows may launch now: it waits for this grid's completion, as this
  // one does for the kernel before it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CastState cs = cast_begin(a.cast);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n_out = kGated ? a.N_in / 2 : a.N_in;
  const int64_t strips = (n_out + kCols - 1) / kCols;
  const int64_t chunk = blockIdx.x / strips, strip = blockIdx.x % strips;
  const int64_t c0 = strip * kCols, col = c0 + lane * 8;
  const int64_t r0 = chunk * kRows;
  int rows = int(a.M - r0 < kRows ? a.M - r0 : kRows);
  asm volatile("" : "+r"(rows));  // every row's address goes by it, so that no row is loaded before this place
  const int64_t groups = scale_groups(TE_MXFP8, a.N_in);
  const uint8_t* scales = static_cast<const uint8_t*>(a.scales) + chunk * groups * 512;
  // the first rows are under way while the scales are fetched
  struct Rows {
    Dy8<T> dy[U];
    uint2 g[U], l[kGated ? U : 1];
  } next;
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes);
  if (col < n_out) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t r = r0 + min(warp + j * kWarps, rows - 1);
      next.dy[j].load(a.dy, r * n_out + col);
      next.g[j] = load8(codes + r * a.N_in + col);
      if constexpr (kGated) next.l[j] = load8(codes + r * a.N_in + n_out + col);
    }
  }
#pragma unroll
  for (int h = 0; h < (kGated ? 2 : 1); ++h)
    for (int i = threadIdx.x; i < kRows * kSb; i += kWarps * 32) {
      const int64_t b = (h * n_out + c0) / 32 + i % kSb;
      const bool in = c0 + i % kSb * 32 < n_out;  // n_out is a multiple of 32
      sc[h][i / kSb][i % kSb] = in ? e8m0_value(scales[scale_offset_wide(i / kSb, b)]) : 0.0f;
    }
  __syncthreads();
  f32x2 acc[kGated ? 2 : 1][4];
  float am[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    acc[0][p] = f2s(0.0f);
    if constexpr (kGated) acc[1][p] = f2s(0.0f);
    am[p] = 0.0f;
  }
  if (col < n_out) {
    with_out_amax(out_kind(cs), a.cast.amax_out != nullptr, [&](auto tag, auto atag) {
      constexpr int OUT = decltype(tag)::value;
      constexpr bool AMAX = decltype(atag)::value;
      auto load = [&](Rows& b, int rb) {  // rows past the end re-read the last
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int64_t r = r0 + min(rb + j * kWarps, rows - 1);
          b.dy[j].load(a.dy, r * n_out + col);
          b.g[j] = load8(codes + r * a.N_in + col);
          if constexpr (kGated) b.l[j] = load8(codes + r * a.N_in + n_out + col);
        }
      };
#pragma unroll 1
      for (int rb = warp; rb < rows; rb += U * kWarps) {
        const Rows cur = next;
        load(next, rb + U * kWarps);  // the next rows are under way while these are computed
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int rl = rb + j * kWarps;
          if (rl >= rows) break;
          const int64_t r = r0 + rl;
          f32x2 d[4], h[4], y[4], g[4];
          float v[8];
          cur.dy[j].get(d);
          decode8(cur.g[j], sc[0][rl][lane >> 2], h);
          if constexpr (kGated) {
            f32x2 l[4], gl[4];
            decode8(cur.l[j], sc[1][rl][lane >> 2], l);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              f32x2 b, db;
              act_both<kBase>(h[p], b, db);
              g[p] = mul2(mul2(d[p], l[p]), db);
              gl[p] = mul2(d[p], b);
              y[p] = mul2(b, l[p]);
              acc[0][p] = add2(acc[0][p], g[p]);
              acc[1][p] = add2(acc[1][p], gl[p]);
              if (AMAX) am[p] = absmax2(absmax2(am[p], g[p]), gl[p]);
            }
            flat8(g, v);
            store_out<OUT, 8>(a.dx, r * a.N_in + col, v, cs);
            flat8(gl, v);
            store_out<OUT, 8>(a.dx, r * a.N_in + n_out + col, v, cs);
          } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              f32x2 db;
              act_both<kBase>(h[p], y[p], db);
              g[p] = mul2(d[p], db);
              acc[0][p] = add2(acc[0][p], g[p]);
              if (AMAX) am[p] = absmax2(am[p], g[p]);
            }
            flat8(g, v);
            store_out<OUT, 8>(a.dx, r * a.N_in + col, v, cs);
          }
          if (a.act_out) {
            flat8(y, v);
            store_out<kPlain, 8>(a.act_out, r * n_out + col, v, cs);
          }
        }
      }
    });
  }
  if (a.dbias) {
#pragma unroll
    for (int h = 0; h < (kGated ? 2 : 1); ++h)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        red[warp][h][lane * 8 + 2 * p] = f2lo(acc[h][p]);
        red[warp][h][lane * 8 + 2 * p + 1] = f2hi(acc[h][p]);
      }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < (kGated ? 2 : 1); ++h) {
      const int j = threadIdx.x;  // kCols threads
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += red[w][h][j];
      if (c0 + j < n_out) a.partials[chunk * a.N_in + h * n_out + c0 + j] = sum;
    }
  }
  block_amax_commit(fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3])), a.cast.amax_out);
}

template <typename T>
te_status launch_t(const DactCkptArgs& a, unsigned grid, cudaStream_t s) {
  const dim3 g(grid), b(kWarps * 32);
  switch (a.act) {
    case TE_RELU: return launch_dependent(dact_ckpt_kernel<T, TE_RELU>, g, b, s, a);
    case TE_GELU: return launch_dependent(dact_ckpt_kernel<T, TE_GELU>, g, b, s, a);
    case TE_SILU: return launch_dependent(dact_ckpt_kernel<T, TE_SILU>, g, b, s, a);
    case TE_SWIGLU: return launch_dependent(dact_ckpt_kernel<T, TE_SWIGLU>, g, b, s, a);
    case TE_GEGLU: return launch_dependent(dact_ckpt_kernel<T, TE_GEGLU>, g, b, s, a);
    default: return launch_dependent(dact_ckpt_kernel<T, TE_REGLU>, g, b, s, a);
  }
}

}  // namespace

te_status launch_dact_ckpt(const DactCkptArgs& args, cudaStream_t s) {
  if (args.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_DACT_DBIAS, s);
  DactCkptArgs a = args;
  const int64_t n_out = is_gated(a.act) ? a.N_in / 2 : a.N_in;
  const int64_t chunks = ceil_div(a.M, kRows), grid = chunks * ceil_div(n_out, kCols);
  if (grid > 0x7fffffff) return TE_ERR_UNSUPPORTED;
  // One row of CTAs: its partial row is the sum (64 x 512 fp32 6.2 us against 7.2 with a second kernel, and
  // 2 us less of the host).  A cluster that added up two to eight of them was no faster for 256 rows and
  // slower for more, as it waits for that many free places at once: 512 x 28672 swiglu 36 us against 30.
  if (chunks == 1) a.partials = a.dbias;
  const te_status st = a.dtype == TE_BF16 ? launch_t<__nv_bfloat16>(a, unsigned(grid), s)
                                          : launch_t<float>(a, unsigned(grid), s);
  if (st != TE_OK || !a.dbias || chunks == 1) return st;
  return launch_colsum(a.partials, int(chunks), a.N_in, a.dbias, s);
}

}  // namespace te

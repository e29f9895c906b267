// The gradient of a dense layer's residual epilogue, out = a * residual + gate * act(z) + ...: one
// pass over dout and z gives dz (the operand of the layer's two products), a * dout, and the column
// sums behind dbias and dgate.  Bound by memory: it reads and writes each tensor once.
//
// A CTA takes a strip of 256 columns (8 to a lane) and a chunk of rows that share a gate, as many as put
// one wave of CTAs on the SMs (in chunks of 128 rows 4100 x 4096 took a second, almost empty one: 35 us
// with gelu, not 21); its 8 warps take the rows in turn, keep the columns' sums in registers, and leave
// one row of partial sums, which a second kernel adds in a fixed order.
#include "cast.cuh"
#include "common.cuh"
#include "kernels.h"

namespace te {

namespace {

constexpr int kWarps = 8;
constexpr int kCtasPerSm = 2;
constexpr int kMaxRows = 256;  // of a chunk: no sum of a thread runs over more than 32
constexpr int kUnroll = 4;  // rows of loads in flight per warp (86 us a call for 89 with 3 CTAs and 2 rows)
constexpr int kStrip = 256;
constexpr int64_t kMaxCols = int64_t(65535) * kStrip;  // of one launch

template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, uint4 (&w)[2]) {
  if constexpr (sizeof(T) == 2) {
    w[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
    w[0] = p[0];
    w[1] = p[1];
  }
}
template <typename T>
__device__ __forceinline__ void cvt8(const uint4 (&w)[2], f32x2 (&p)[4]) {
  if constexpr (sizeof(T) == 2) {
    Pairs<__nv_bfloat16>::cvt(w[0], p);
  } else {
    f32x2 a[2], b[2];
    Pairs<float>::cvt(w[0], a);
    Pairs<float>::cvt(w[1], b);
    p[0] = a[0]; p[1] = a[1]; p[2] = b[0]; p[3] = b[1];
  }
}

// Two bf16 values, but no less than lo and no more than hi; a NaN stays one.
__device__ __forceinline__ uint32_t above(uint32_t w, uint32_t lo) {
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(lo));
  return w;
}
__device__ __forceinline__ uint32_t below(uint32_t w, uint32_t hi) {
  asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(hi));
  return w;
}

// An activation and its derivative at two bf16 values.
// gelu(h) = h s and gelu'(h) = s + 2 h sqrt(2/pi) (1 + 3 * 0.044715 h^2) s (1 - s) from one logistic
// s = 1 / (1 + e) of twice the inner function, 1 - s = e s; silu(h) = h s and silu'(h) = s (1 + h (1 - s)) likewise.
// h is held where s still moves: from below, so that e stays finite (at -9.875 and -80 s is under 2^-115), and for
// all but the product h s from above, where the powers of h would overflow against 1 - s = 0.
template <int ACT>
__device__ __forceinline__ void act_both(uint32_t w, f32x2& act, f32x2& dact) {
  if constexpr (ACT == TE_GELU) {
    w = above(w, 0xC11EC11Eu);
    const f32x2 h = bf16x2_f2(w), c = bf16x2_f2(below(w, 0x41804180u)), cc = mul2(c, c);  // 16
    const f32x2 e = ex2_2(mul2(c, fma2(cc, f2s(kGeluA2), f2s(kGeluA1))));
    const f32x2 s = rcp2(add2(e, f2s(1.0f)));
    const f32x2 q = mul2(c, fma2(cc, f2s(6.0f * kGeluK0 * kGeluK1), f2s(2.0f * kGeluK0)));
    act = mul2(h, s);
    dact = fma2(q, mul2(s, mul2(e, s)), s);
  } else if constexpr (ACT == TE_SILU) {
    w = above(w, 0xC2A0C2A0u);
    const f32x2 h = bf16x2_f2(w), c = bf16x2_f2(below(w, 0x43004300u));  // 128
    const f32x2 e = ex2_2(mul2(c, f2s(-kLog2e)));
    const f32x2 s = rcp2(add2(e, f2s(1.0f)));
    act = mul2(h, s);
    dact = mul2(s, fma2(c, mul2(e, s), f2s(1.0f)));
  } else {
    const f32x2 h = bf16x2_f2(w);
    act = act2c<ACT>(h);
    dact = dact2c<ACT>(h);
  }
}

// Rows of a chunk, and the chunks of one gate's rows.
int64_t rows_of(int64_t M, int64_t N, int64_t gate_rows) {
  const int64_t chunks = int64_t(num_sms()) * kCtasPerSm / ceil_div(N, int64_t(kStrip));
  int64_t per_gate = chunks / (M / gate_rows);
  if (per_gate < 1) per_gate = 1;
  per_gate *= ceil_div(gate_rows, per_gate * kMaxRows);  // (whole waves of shorter chunks)
  const int64_t rows = ceil_div(gate_rows, per_gate);
  return (rows + kWarps - 1) / kWarps * kWarps;  // whole rounds of the warps
}
__host__ __device__ __forceinline__ int64_t chunks_of(int64_t gate_rows, int64_t rows) {
  return (gate_rows + rows - 1) / rows;
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) dense_residual_grad_kernel(DenseResidualGradArgs a) {
  __shared__ float red[kWarps][2][kStrip];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CastState cs = cast_begin(a.cast);
  const int kind = a.dz ? out_kind(cs) : int(OUT_NONE);
  const bool want_amax = a.cast.amax_out != nullptr;
  const bool read_z = ACT != TE_IDENTITY || a.dgate != nullptr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t(blockIdx.y) * 32 + lane) * 8;
  const int64_t per_gate = chunks_of(a.gate_rows, a.chunk_rows);
  const int64_t gate_row = blockIdx.x / per_gate;
  const int64_t r0 = gate_row * a.gate_rows + (blockIdx.x % per_gate) * a.chunk_rows;
  const int64_t end = (gate_row + 1) * a.gate_rows;
  const int64_t r1 = r0 + a.chunk_rows < end ? r0 + a.chunk_rows : end;
  f32x2 sz[4], sa[4], gt[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) sz[p] = sa[p] = f2s(0.0f), gt[p] = f2s(1.0f);
  float amax = 0.0f;
  if (col < a.cols) {
    if (a.gate) Pairs<__nv_bfloat16>::cvt(__ldg(reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(a.gate) + gate_row * a.N + col)), gt);
    for (int64_t rb = r0 + warp; rb < r1; rb += kUnroll * kWarps) {
      uint4 d[kUnroll][2], z[kUnroll][2];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int64_t r = rb + j * kWarps;
        d[j][0] = d[j][1] = z[j][0] = z[j][1] = make_uint4(0u, 0u, 0u, 0u);
        if (r < r1) {
          load8<T>(a.dout, r * a.N + col, d[j]);
          if (read_z) load8<__nv_bfloat16>(a.z, r * a.N + col, z[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int64_t r = rb + j * kWarps;
        if (r >= r1) break;
        const int64_t at = r * a.N + col;
        f32x2 dp[4];
        cvt8<T>(d[j], dp);
        const uint32_t zw[4] = {z[j][0].x, z[j][0].y, z[j][0].z, z[j][0].w};
        float o[8], s[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          s[2 * p] = a.residual_scale * f2lo(dp[p]);
          s[2 * p + 1] = a.residual_scale * f2hi(dp[p]);
          f32x2 act, dact;
          act_both<ACT>(zw[p], act, dact);
          sa[p] = fma2(dp[p], act, sa[p]);
          f32x2 v = ACT == TE_IDENTITY ? dp[p] : mul2(dp[p], dact);
          v = mul2(v, gt[p]);
          sz[p] = add2(sz[p], v);
          if (want_amax) amax = absmax2(amax, v);
          o[2 * p] = f2lo(v);
          o[2 * p + 1] = f2hi(v);
        }
        if (kind == OUT_BF16) store_out<OUT_BF16, 8>(a.dz, at, o, cs);
        else if (kind == OUT_E4M3) store_out<OUT_E4M3, 8>(a.dz, at, o, cs);
        if (a.dresidual) store_out<(sizeof(T) == 2 ? OUT_BF16 : OUT_F32), 8>(a.dresidual, at, s, cs);
      }
    }
  }
  if (a.dbias || a.dgate) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      red[warp][0][lane * 8 + 2 * p] = f2lo(sz[p]);
      red[warp][0][lane * 8 + 2 * p + 1] = f2hi(sz[p]);
      red[warp][1][lane * 8 + 2 * p] = f2lo(sa[p]);
      red[warp][1][lane * 8 + 2 * p + 1] = f2hi(sa[p]);
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * kStrip; t += blockDim.x) {
      const int h = t / kStrip, j = t % kStrip;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += red[w][h][j];
      const int64_t c = int64_t(blockIdx.y) * kStrip + j;
      if (c < a.cols && (h == 0 ? a.dbias != nullptr : a.dgate != nullptr))
        a.partials[(int64_t(blockIdx.x) * 2 + h) * a.N + c] = sum;
    }
  }
  if (a.cast.amax_out) {
    amax = warp_max(amax);
    if (lane == 0) atomic_max_nonneg(a.cast.amax_out, amax);
  }
}

// dbias (blockIdx.y = 0) and the rows of dgate (1 and up, a grid's stride apart): the partial rows of
// all chunks, or of one gate's.  A CTA takes 128 columns, four to a lane; its warps take every 16th
// chunk and are added in warp order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) dense_residual_sum_kernel(DenseResidualGradArgs a, int64_t gates) {
  __shared__ float4 sums[kSumWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t j = int64_t(blockIdx.x) * 128 + lane * 4;  // N is a multiple of 16
  const int64_t per_gate = chunks_of(a.gate_rows, a.chunk_rows);
  auto column = [&](int64_t c0, int64_t c1, int half, float* out) {
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j < a.N) {
#pragma unroll 4
      for (int64_t c = c0 + w; c < c1; c += kSumWarps) {
        const float4 v = *reinterpret_cast<const float4*>(a.partials + (c * 2 + half) * a.N + j);
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
      }
    }
    __syncthreads();
    sums[w][lane] = t;
    __syncthreads();
    if (w == 0 && j < a.N) {
      for (int k = 1; k < kSumWarps; ++k) {
        const float4 v = sums[k][lane];
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
      }
      out[j] = t.x; out[j + 1] = t.y; out[j + 2] = t.z; out[j + 3] = t.w;
    }
  };
  if (blockIdx.y == 0) {
    if (a.dbias) column(0, gates * per_gate, 0, a.dbias);
    return;
  }
  for (int64_t g = int64_t(blockIdx.y) - 1; g < gates; g += int64_t(gridDim.y) - 1)
    column(g * per_gate, (g + 1) * per_gate, 1, a.dgate + g * a.N);
}

template <typename T>
void launch_act(const DenseResidualGradArgs& a, dim3 grid, cudaStream_t s) {
  switch (a.act) {
    case TE_RELU: dense_residual_grad_kernel<T, TE_RELU><<<grid, kWarps * 32, 0, s>>>(a); break;
    case TE_GELU: dense_residual_grad_kernel<T, TE_GELU><<<grid, kWarps * 32, 0, s>>>(a); break;
    case TE_SILU: dense_residual_grad_kernel<T, TE_SILU><<<grid, kWarps * 32, 0, s>>>(a); break;
    default: dense_residual_grad_kernel<T, TE_IDENTITY><<<grid, kWarps * 32, 0, s>>>(a); break;
  }
}

}  // namespace

size_t dense_residual_grad_workspace(int64_t M, int64_t N, int64_t gates) {
  if (M <= 0 || N <= 0) return 0;
  if (gates < 1 || gates > M) gates = 1;
  const int64_t gate_rows = M / gates;
  return size_t(chunks_of(gate_rows, rows_of(M, N, gate_rows)) * gates) * 2 * size_t(N) * sizeof(float);
}

te_status launch_dense_residual_grad(DenseResidualGradArgs a, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_DACT_DBIAS, s);
  a.chunk_rows = rows_of(a.M, a.N, a.gate_rows);
  const int64_t gates = a.M / a.gate_rows, chunks = gates * chunks_of(a.gate_rows, a.chunk_rows);
  // Strips go along y, whose size is limited: what lies behind it in another launch.  (One dimension, taken apart
  // in the kernel, or a first strip among the arguments cost 8% at 16384 x 8192: the kernel needs every register.)
  for (int64_t at = 0; at < a.N; at += kMaxCols) {
    DenseResidualGradArgs b = a;
    auto from = [&](auto* p, size_t es) { return p ? reinterpret_cast<decltype(p)>(uintptr_t(p) + size_t(at) * es) : p; };
    const size_t es = a.dtype == TE_F32 ? 4 : 2;
    b.dout = from(a.dout, es);
    b.dresidual = from(a.dresidual, es);
    b.z = from(a.z, 2);
    b.gate = from(a.gate, 2);
    b.dz = from(a.dz, a.cast.out_dtype == TE_E4M3 ? 1 : 2);
    b.partials = from(a.partials, 4);
    b.cols = a.N - at < kMaxCols ? a.N - at : kMaxCols;
    const dim3 grid{unsigned(chunks), unsigned(ceil_div(b.cols, kStrip))};
    if (a.dtype == TE_F32) launch_act<float>(b, grid, s);
    else launch_act<__nv_bfloat16>(b, grid, s);
  }
  if (cudaGetLastError() != cudaSuccess) return TE_ERR_CUDA;
  if (!a.dbias && !a.dgate) return TE_OK;
  const int64_t rows = a.dgate ? 1 + (gates < 1024 ? gates : 1024) : 1;
  return launch_dependent(dense_residual_sum_kernel, dim3(unsigned(ceil_div(a.N, 128)), unsigned(rows)),
                          dim3(kSumWarps * 32), s, a, gates);
}

}  // namespace te

// C entry points of the block-scaled operators: argument checks, workspace carving and the order
// of the kernels on the caller's stream.  The contract of each is in include/te_gb300.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_util.h"
#include "kernels.h"
#include "te_gb300.h"

namespace te {
namespace {

bool valid_format(int f) { return f >= TE_MXFP8 && f <= TE_NVFP4; }
bool valid_fp4(int f) { return f == TE_MXFP4 || f == TE_NVFP4; }
bool valid_norm_dims(int64_t M, int64_t a, int64_t b) { return M >= 0 && a > 0 && b > 0; }

// A quantizer is the tensor scale of NVFP4; the MX formats have none.
bool format_quantizer_ok(int f, const te_quantizer* q) {
  return f == TE_NVFP4 ? enabled(q) && quantizer_ok(q) : q == nullptr;
}

// A product's quantizer writes its factor and its amax, with current scaling its scale too: none of
// them can be the factor of an operand packed before.
bool factor_ok(const te_quantizer* q, const float* other) {
  if (!q) return true;
  if (!q->scale_inv) return false;
  return !other || (q->scale_inv != other && q->amax != other &&
                    (q->mode != TE_SCALING_CURRENT || q->scale != other));
}

// Gives a its tensor scale's places; NVFP4 finds this call's amax first when the scale is to come
// from it.
te_status take_tensor_scale(BlockQuantArgs& a, const te_quantizer* q, cudaStream_t s) {
  if (a.fmt == TE_NVFP4) {
    if (q->mode == TE_SCALING_CURRENT) {
      const te_status st = launch_amax(a.x, a.x_dtype, a.M * a.N, q->amax, s);
      if (st != TE_OK) return st;
      a.amax_in = q->amax;
      a.scale_out = q->scale;
    } else {
      const te_status st = zero_scalar(q->amax, s);
      if (st != TE_OK) return st;
      a.scale = q->scale;
      a.amax_out = q->amax;
    }
    a.scale_inv_out = q->scale_inv;
  }
  return TE_OK;
}

te_status block_quantize(BlockQuantArgs a, const te_quantizer* q, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  const te_status st = take_tensor_scale(a, q, s);
  return st == TE_OK ? launch_block_quantize(a, s) : st;
}

// A packed tensor in the workspace, large enough for either 4-bit format.
struct Packed {
  void* codes;
  void* scales;
};
Packed take_packed(Carver& c, int64_t rows, int64_t cols) {
  Packed p;
  p.codes = c.take(size_t(rows) * size_t(cols) / 2);
  p.scales = c.take(block_scale_bytes(TE_NVFP4, rows, cols));
  return p;
}

struct DenseFp4Bwd {
  Packed dy, dyt;
  int64_t pitch;  // bytes from one row of dyt to the next
  float* partials;
  size_t bytes;
};

DenseFp4Bwd dense_fp4_bwd_layout(void* ws, int64_t M, int64_t N) {
  Carver c(ws);
  DenseFp4Bwd L;
  L.dy = take_packed(c, M, N);
  // Rows that begin on 64 bytes: the TMA engine's 128-byte reads of others touch a line more, which
  // costs a product with two such operands up to a quarter of its time (4096 x 16384 x 4128: 110 us;
  // with 4224 codes a row 89).  x^T comes as the caller has it; a copy of it costs what it gains.
  L.pitch = (pad32(M) / 2 + 63) / 64 * 64;
  L.dyt.codes = c.take(size_t(N) * size_t(L.pitch));
  L.dyt.scales = c.take(block_scale_bytes(TE_NVFP4, N, pad32(M)));
  L.partials = static_cast<float*>(c.take(dact_dbias_workspace(M, N)));
  L.bytes = c.used;
  return L;
}

}  // namespace

size_t dense_fp4_fwd_workspace(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  Carver c(nullptr);
  take_packed(c, M, K);
  return c.used;
}

size_t dense_fp4_bwd_workspace(int64_t M, int64_t N) {
  return M <= 0 || N <= 0 ? 0 : dense_fp4_bwd_layout(nullptr, M, N).bytes;
}

}  // namespace te

using namespace te;

extern "C" {

size_t te_block_scale_bytes(te_block_format format, int64_t rows, int64_t cols) {
  if (!valid_format(format) || rows < 0 || cols < 0) return 0;
  return block_scale_bytes(format, rows, cols);
}

te_status te_block_quantize(const void* x, te_dtype x_dtype, int64_t M, int64_t N,
                            te_block_format format, const te_quantizer* q, void* codes,
                            void* scales, void* codes_t, void* scales_t, void* stream) {
  if (M < 0 || N <= 0 || !is_act_dtype(x_dtype) || !valid_format(format) ||
      !format_quantizer_ok(format, q) || !codes != !scales || !codes_t != !scales_t ||
      (M > 0 && (!x || (!codes && !codes_t))))
    return TE_ERR_INVALID_ARG;
  if (N % (codes ? 32 : 16) || (codes_t && format == TE_MXFP8)) return TE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(codes_t) ||
      !aligned16(scales_t))
    return TE_ERR_UNSUPPORTED;
  BlockQuantArgs a;
  a.x = x;
  a.x_dtype = x_dtype;
  a.M = M;
  a.N = N;
  a.fmt = format;
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  return block_quantize(a, q, as_stream(stream));
}

te_status te_block_dequantize(const void* codes, const void* scales, te_block_format format,
                              const float* scale_inv, int64_t M, int64_t N, void* out,
                              te_dtype out_dtype, void* stream) {
  if (M < 0 || N <= 0 || !is_act_dtype(out_dtype) || !valid_format(format) ||
      (scale_inv && format != TE_NVFP4) || (M > 0 && (!codes || !scales || !out)))
    return TE_ERR_INVALID_ARG;
  if (N % 32 || !aligned16(codes) || !aligned16(scales) || !aligned16(out) || !aligned4(scale_inv))
    return TE_ERR_UNSUPPORTED;
  BlockDequantArgs a;
  a.codes = codes;
  a.scales = scales;
  a.fmt = format;
  a.scale_inv = scale_inv;
  a.M = M;
  a.N = N;
  a.out = out;
  a.out_dtype = out_dtype;
  return launch_block_dequantize(a, as_stream(stream));
}

te_status te_block_gemm(const void* A, const void* a_scales, const void* B, const void* b_scales,
                        te_block_format format, int64_t M, int64_t N, int64_t K,
                        const float* a_scale_inv, const float* b_scale_inv, const void* bias,
                        te_dtype bias_dtype, void* D, te_dtype d_dtype, void* stream) {
  if (!valid_norm_dims(M, N, K) || !valid_format(format) || !is_act_dtype(d_dtype) ||
      (bias && !is_act_dtype(bias_dtype)) ||
      (M > 0 && (!A || !a_scales || !B || !b_scales || !D)))
    return TE_ERR_INVALID_ARG;
  if (!valid_fp4(format) || N % 16 || K % 32) return TE_ERR_UNSUPPORTED;
  if (!aligned16(A) || !aligned16(a_scales) || !aligned16(B) || !aligned16(b_scales) ||
      !aligned16(D) || !opt_aligned16(bias) || !aligned4(a_scale_inv) || !aligned4(b_scale_inv))
    return TE_ERR_UNSUPPORTED;
  BlockGemmArgs g;
  g.A = A;
  g.a_scales = a_scales;
  g.B = B;
  g.b_scales = b_scales;
  g.fmt = format;
  g.M = M;
  g.N = N;
  g.K = K;
  g.a_scale_inv = a_scale_inv;
  g.b_scale_inv = b_scale_inv;
  g.bias = bias;
  g.bias_dtype = bias_dtype;
  g.D = D;
  g.d_dtype = d_dtype;
  return launch_block_gemm(g, as_stream(stream));
}

te_status te_dense_fp4_fwd(const void* x, te_dtype dtype, const void* kernel,
                           const void* kernel_scales, te_block_format format,
                           const te_quantizer* q, const float* kernel_scale_inv, const void* bias,
                           int64_t M, int64_t K, int64_t N, void* out, void* saved_xt,
                           void* saved_xt_scales, void* workspace, size_t ws_bytes, void* stream) {
  if (!valid_norm_dims(M, K, N) || !is_act_dtype(dtype) || !valid_format(format) ||
      !format_quantizer_ok(format, q) || !factor_ok(q, kernel_scale_inv) || !saved_xt != !saved_xt_scales ||
      (M > 0 && (!x || !kernel || !kernel_scales || !out)))
    return TE_ERR_INVALID_ARG;
  if (!valid_fp4(format) || K % 32 || N % 16) return TE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(kernel) || !aligned16(kernel_scales) || !opt_aligned16(bias) ||
      !aligned16(out) || !opt_aligned16(saved_xt) || !opt_aligned16(saved_xt_scales) ||
      !aligned16(workspace) || !aligned4(kernel_scale_inv))
    return TE_ERR_UNSUPPORTED;
  if (M == 0) return TE_OK;
  cudaStream_t s = as_stream(stream);
  BlockQuantArgs a;
  a.x = x;
  a.x_dtype = dtype;
  a.M = M;
  a.N = K;
  a.fmt = format;
  BlockGemmArgs g;
  g.B = kernel;
  g.b_scales = kernel_scales;
  g.fmt = format;
  g.M = M;
  g.N = N;
  g.K = K;
  g.b_scale_inv = kernel_scale_inv;
  g.bias = bias;
  g.bias_dtype = dtype;
  g.D = out;
  g.d_dtype = dtype;
  if (M <= kFewPacked && !saved_xt) {
    const te_status st = take_tensor_scale(a, q, s);
    if (st != TE_OK) return st;
    g.b_ready = a.amax_in != nullptr;  // only the search for the amax precedes the product
    return launch_block_gemm_packing(g, a, s);
  }
  Carver c(workspace);
  const Packed xq = take_packed(c, M, K);
  if (!workspace || ws_bytes < c.used) return TE_ERR_WORKSPACE;
  a.codes = xq.codes;
  a.scales = xq.scales;
  a.codes_t = saved_xt;
  a.scales_t = saved_xt_scales;
  const te_status st = block_quantize(a, q, s);
  if (st != TE_OK) return st;
  g.A = xq.codes;
  g.a_scales = xq.scales;
  g.a_scale_inv = q ? q->scale_inv : nullptr;
  g.b_ready = 1;  // only the packing of x lies between the caller's work and this product
  return launch_block_gemm(g, s);
}

te_status te_dense_fp4_bwd(const void* dy, te_dtype dtype, const void* kernel,
                           const void* kernel_scales, const void* saved_xt,
                           const void* saved_xt_scales, te_block_format format,
                           const te_quantizer* q, const float* kernel_scale_inv,
                           const float* x_scale_inv, int64_t M, int64_t K, int64_t N, void* dx,
                           void* dkernel, float* dbias, void* workspace, size_t ws_bytes,
                           void* stream) {
  if (!valid_norm_dims(M, K, N) || !is_act_dtype(dtype) || !valid_format(format) ||
      !format_quantizer_ok(format, q) || !factor_ok(q, kernel_scale_inv) || !factor_ok(q, x_scale_inv) ||
      !dkernel ||
      (M > 0 && (!dy || !kernel || !kernel_scales || !saved_xt || !saved_xt_scales || !dx)))
    return TE_ERR_INVALID_ARG;
  if (!valid_fp4(format) || K % 32 || N % 32) return TE_ERR_UNSUPPORTED;
  if (!aligned16(dy) || !aligned16(kernel) || !aligned16(kernel_scales) || !aligned16(saved_xt) ||
      !aligned16(saved_xt_scales) || !aligned16(dx) || !aligned16(dkernel) || !aligned4(dbias) ||
      !aligned16(workspace) || !aligned4(kernel_scale_inv) || !aligned4(x_scale_inv))
    return TE_ERR_UNSUPPORTED;
  cudaStream_t s = as_stream(stream);
  if (M == 0) {
    if (cudaMemsetAsync(dkernel, 0, size_t(K) * N * esize(dtype), s) != cudaSuccess) return TE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, size_t(N) * 4, s) != cudaSuccess) return TE_ERR_CUDA;
    return TE_OK;
  }
  const DenseFp4Bwd L = dense_fp4_bwd_layout(workspace, M, N);
  if (!workspace || ws_bytes < L.bytes) return TE_ERR_WORKSPACE;
  BlockQuantArgs a;
  a.x = dy;
  a.x_dtype = dtype;
  a.M = M;
  a.N = N;
  a.fmt = format;
  a.codes = L.dy.codes;
  a.scales = L.dy.scales;
  a.codes_t = L.dyt.codes;
  a.scales_t = L.dyt.scales;
  a.pitch_t = L.pitch;
  a.partials = dbias ? L.partials : nullptr;
  te_status st = block_quantize(a, q, s);
  if (st != TE_OK) return st;
  if (dbias) {
    st = launch_colsum(L.partials, int((M + 127) / 128), N, dbias, s);
    if (st != TE_OK) return st;
  }
  // dx = dy kernel^T (contraction over N)
  BlockGemmArgs g;
  g.A = L.dy.codes;
  g.a_scales = L.dy.scales;
  g.B = kernel;
  g.b_scales = kernel_scales;
  g.fmt = format;
  g.M = M;
  g.N = K;
  g.K = N;
  g.a_scale_inv = q ? q->scale_inv : nullptr;
  g.b_scale_inv = kernel_scale_inv;
  g.D = dx;
  g.d_dtype = dtype;
  st = launch_block_gemm(g, s);
  if (st != TE_OK) return st;
  // dkernel = x^T dy (contraction over the rows, filled up with zeros)
  BlockGemmArgs w;
  w.A = saved_xt;
  w.a_scales = saved_xt_scales;
  w.B = L.dyt.codes;
  w.b_scales = L.dyt.scales;
  w.fmt = format;
  w.M = K;
  w.N = N;
  w.K = pad32(M);
  w.b_pitch = L.pitch;
  w.a_scale_inv = x_scale_inv;
  w.b_scale_inv = q ? q->scale_inv : nullptr;
  w.D = dkernel;
  w.d_dtype = dtype;
  return launch_block_gemm(w, s);
}

te_status te_dact_dbias_ckpt(const void* dy, const void* codes, const void* scales, te_dtype dtype,
                             int64_t M, int64_t N_in, te_act_type act, const te_quantizer* q,
                             void* dx, te_dtype dx_dtype, void* act_out, float* dbias,
                             void* workspace, size_t ws_bytes, void* stream) {
  if (M < 0 || N_in <= 0 || !is_act_dtype(dtype) || act == TE_IDENTITY || !valid_act(act) ||
      dx_dtype < TE_F32 || dx_dtype > TE_E4M3)
    return TE_ERR_INVALID_ARG;
  if (M > 0 && (!dy || !codes || !scales || !dx)) return TE_ERR_INVALID_ARG;
  if (dx_dtype == TE_E4M3 && !enabled(q)) return TE_ERR_INVALID_ARG;
  if (!quantizer_ok(q)) return TE_ERR_INVALID_ARG;
  const int64_t n_out = is_gated(act) ? N_in / 2 : N_in;
  if ((is_gated(act) && N_in % 2) || n_out % 32) return TE_ERR_UNSUPPORTED;
  if (!aligned16(dy) || !aligned16(codes) || !aligned16(scales) || !aligned16(dx) ||
      !opt_aligned16(act_out) || !aligned4(dbias))
    return TE_ERR_UNSUPPORTED;
  cudaStream_t s = as_stream(stream);
  if (dbias && M == 0)
    return cudaMemsetAsync(dbias, 0, size_t(N_in) * 4, s) == cudaSuccess ? TE_OK : TE_ERR_CUDA;
  if (M == 0) return TE_OK;
  if (dbias && (!workspace || ws_bytes < dact_dbias_workspace(M, N_in))) return TE_ERR_WORKSPACE;
  if (dbias && !aligned16(workspace)) return TE_ERR_UNSUPPORTED;
  DactCkptArgs a;
  a.dy = dy;
  a.codes = codes;
  a.scales = scales;
  a.dtype = dtype;
  a.M = M;
  a.N_in = N_in;
  a.act = act;
  a.dx = dx;
  a.partials = static_cast<float*>(workspace);
  return dact_ckpt_cast(a, dx_dtype == TE_E4M3 ? q : nullptr, dx_dtype, act_out, dbias, s);
}

}  // extern "C"

// C entry points of the operators around the residual stream: the norms before and after a block, the
// dense layer that ends in the stream, and the norm and clipping of gradients.  Checks of arguments
// and the composition of the kernels; the contract of each is in include/te_gb300.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "api_util.h"
#include "common.cuh"
#include "kernels.h"
#include "te_gb300.h"

namespace te {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;  // rows and columns (the products' tile arithmetic)

// Memory that a call reads and writes.  clash() is whether something written overlaps anything else
// (a tensor that may be updated in place is added as written only).
class Spans {
 public:
  void reads(const void* p, size_t bytes) { add(p, bytes, false); }
  void writes(const void* p, size_t bytes) { add(p, bytes, true); }
  // the factors of a quantizer
  void quantizer(const te_quantizer* q) {
    if (!q) return;
    if (q->mode == TE_SCALING_CURRENT) writes(q->scale, 4);
    else reads(q->scale, 4);
    writes(q->scale_inv, 4);
    writes(q->amax, 4);
  }
  bool clash() const {
    for (int i = 0; i < n_; ++i)
      for (int j = i + 1; j < n_; ++j)
        if ((s_[i].out || s_[j].out) && s_[i].lo < s_[j].hi && s_[j].lo < s_[i].hi) return true;
    return false;
  }

 private:
  struct Span {
    uintptr_t lo, hi;
    bool out;
  };
  void add(const void* p, size_t bytes, bool out) {
    if (p && bytes) s_[n_++] = Span{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, out};
  }
  Span s_[32];
  int n_ = 0;
};

bool valid_norm(int t) { return t == TE_LAYERNORM || t == TE_RMSNORM; }
// Types of the block's tensors and of the stream.
bool valid_stream(int dtype, int residual_dtype) {
  return (dtype == TE_BF16 && is_act_dtype(residual_dtype)) || (dtype == TE_F32 && residual_dtype == TE_F32);
}
// Rows of a gate (1 without one, or without rows), or 0 for a bad number of gates.
int64_t gate_rows_of(const void* gate, int64_t gates, int64_t M) {
  if (!gate) return M > 0 ? M : 1;
  if (gates < 1 || M % gates) return 0;
  return M > 0 ? M / gates : 1;
}

te_status zero(void* p, size_t bytes, cudaStream_t s) {
  if (!p || !bytes) return TE_OK;
  return cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

size_t dense_fwd_workspace(int64_t M, int64_t K, int64_t N, int dtype) {
  return dense_few_serves(M, N, K, dtype) ? 0 : gemm_split_workspace(M, N, K, dtype, EPI_RESIDUAL);
}

struct DenseBwdLayout {
  float* partials = nullptr;
  void* dz = nullptr;
  SplitScratch split;
  size_t bytes = 0;
};
DenseBwdLayout dense_bwd_layout(void* ws, int64_t M, int64_t K, int64_t N, int64_t gates, int dtype) {
  Carver c(ws);
  DenseBwdLayout L;
  L.partials = static_cast<float*>(c.take(dense_residual_grad_workspace(M, N, gates)));
  L.dz = c.take(size_t(M) * N * esize(dtype));
  L.split = carve_split(c, {gemm_split_workspace(M, K, N, dtype, EPI_BIAS), gemm_split_workspace(K, N, M, dtype, EPI_BIAS)});
  L.bytes = c.used;
  return L;
}

te_status check_grads(const te_grad* grads, int64_t n, bool clip, const float* norm, const void* ws, size_t ws_bytes,
                      std::vector<GradTensor>* out) {
  if (n < 0 || (n > 0 && !grads) || !norm) return TE_ERR_INVALID_ARG;
  struct Span {
    uintptr_t lo, hi;
  };
  std::vector<Span> in, written;
  written.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4});
  for (int64_t i = 0; i < n; ++i) {
    GradTensor g = grads[i];
    if (g.numel < 0 || !is_act_dtype(g.dtype) || (g.numel > 0 && !g.data)) return TE_ERR_INVALID_ARG;
    if (!g.out) g.out = const_cast<void*>(g.data);
    const size_t es = esize(g.dtype);
    if (reinterpret_cast<uintptr_t>(g.data) % es || (clip && reinterpret_cast<uintptr_t>(g.out) % es))
      return TE_ERR_UNSUPPORTED;
    if (g.numel > kMaxDim * kMaxDim / 16) return TE_ERR_UNSUPPORTED;
    if (g.numel == 0) continue;
    const size_t bytes = size_t(g.numel) * es;
    const uintptr_t p = reinterpret_cast<uintptr_t>(g.data), o = reinterpret_cast<uintptr_t>(g.out);
    if (!clip || o != p) in.push_back({p, p + bytes});
    if (clip) written.push_back({o, o + bytes});
    out->push_back(g);
  }
  if (!aligned4(norm)) return TE_ERR_UNSUPPORTED;
  if (!out->empty() && ws) {
    const size_t used = std::min(ws_bytes, grad_norm_workspace(n));
    if (used) written.push_back({reinterpret_cast<uintptr_t>(ws), reinterpret_cast<uintptr_t>(ws) + used});
  }
  // what is written overlaps nothing
  auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  for (auto* v : {&in, &written})
    if (!std::is_sorted(v->begin(), v->end(), before)) std::sort(v->begin(), v->end(), before);
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].lo < written[i - 1].hi) return TE_ERR_INVALID_ARG;
  // (reads may overlap one another: each is held against the first written span that ends behind its start)
  size_t w = 0;
  for (const Span& s : in) {
    while (w < written.size() && written[w].hi <= s.lo) ++w;
    if (w < written.size() && written[w].lo < s.hi) return TE_ERR_INVALID_ARG;
  }
  if (!out->empty() && (!ws || ws_bytes < grad_norm_workspace(n))) return TE_ERR_WORKSPACE;
  if (!aligned16(ws)) return TE_ERR_UNSUPPORTED;
  return TE_OK;
}

te_status grads(const te_grad* g, int64_t n, bool clip, double max_norm, double epsilon, float* norm, void* ws,
                size_t ws_bytes, cudaStream_t s) {
  try {
    std::vector<GradTensor> t;
    t.reserve(size_t(n > 0 && n < 65536 ? n : 0));
    te_status st = check_grads(g, n, clip, norm, ws, ws_bytes, &t);
    if (st != TE_OK) return st;
    if (t.empty()) return zero(norm, sizeof(float), s);
    GradSlot* slots = static_cast<GradSlot*>(ws);
    int used = 0;
    st = launch_grad_squares(t.data(), int64_t(t.size()), slots, &used, s);
    if (st != TE_OK) return st;
    return clip ? launch_grad_clip(t.data(), int64_t(t.size()), slots, used, max_norm, epsilon, norm, s)
                : launch_grad_norm(slots, used, norm, s);
  } catch (const std::bad_alloc&) {
    return TE_ERR_UNSUPPORTED;
  }
}

}  // namespace
}  // namespace te

using namespace te;

extern "C" {

te_status te_residual_norm_fwd(const void* y, te_dtype dtype, const void* residual, te_dtype residual_dtype, int64_t M,
                               int64_t H, const void* gamma, const void* beta, const void* post_gamma,
                               const void* post_beta, const void* gate, int64_t gates, float residual_scale,
                               te_norm_type norm_type, int zero_centered_gamma, float epsilon, const te_quantizer* q,
                               void* x_out, void* out, te_dtype out_dtype, float* mu, float* rsigma, float* post_mu,
                               float* post_rsigma, void* stream) {
  if (M < 0 || H <= 0 || !valid_stream(dtype, residual_dtype) || out_dtype < TE_F32 || out_dtype > TE_E4M3 ||
      !valid_norm(norm_type))
    return TE_ERR_INVALID_ARG;
  if (M > 0 && (!y || !residual || !gamma || !x_out || !out)) return TE_ERR_INVALID_ARG;
  if (!post_gamma && (post_beta || post_mu || post_rsigma)) return TE_ERR_INVALID_ARG;
  if (norm_type == TE_RMSNORM) beta = post_beta = nullptr;  // not read
  const int64_t gate_rows = gate_rows_of(gate, gates, M);
  if (gate_rows == 0) return TE_ERR_INVALID_ARG;
  if ((out_dtype == TE_E4M3 && !enabled(q)) || !quantizer_ok(q) || (q && !aligned4(q->amax))) return TE_ERR_INVALID_ARG;
  if (H % 8 || H > 8192 || M > kMaxDim) return TE_ERR_UNSUPPORTED;
  for (const void* p : {y, residual, gamma, beta, post_gamma, post_beta, gate, static_cast<const void*>(x_out),
                        static_cast<const void*>(out)})
    if (!aligned16(p)) return TE_ERR_UNSUPPORTED;
  if (!aligned4(mu) || !aligned4(rsigma) || !aligned4(post_mu) || !aligned4(post_rsigma)) return TE_ERR_UNSUPPORTED;
  if (M == 0) return TE_OK;
  const size_t e = esize(dtype), vec = size_t(H) * e, rows = size_t(M) * H, stat = size_t(M) * 4;
  Spans spans;
  spans.reads(y, rows * e);
  if (x_out != residual) spans.reads(residual, rows * esize(residual_dtype));
  for (const void* p : {gamma, beta, post_gamma, post_beta}) spans.reads(p, vec);
  spans.reads(gate, gate ? vec * size_t(gates) : 0);
  spans.writes(x_out, rows * esize(residual_dtype));
  spans.writes(out, rows * esize(out_dtype));
  for (const void* p : {mu, rsigma, post_mu, post_rsigma}) spans.writes(p, stat);
  if (out_dtype == TE_E4M3) spans.quantizer(q);
  else if (q) spans.writes(q->amax, 4);
  if (spans.clash()) return TE_ERR_INVALID_ARG;
  ResidualNormArgs a;
  a.y = y;
  a.residual = residual;
  a.y_dtype = dtype;
  a.residual_dtype = residual_dtype;
  a.M = M;
  a.H = H;
  a.gamma = gamma;
  a.beta = beta;
  a.post_gamma = post_gamma;
  a.post_beta = post_beta;
  a.gate = gate;
  a.gate_rows = gate_rows;
  a.residual_scale = residual_scale;
  a.norm_type = norm_type;
  a.zero_centered_gamma = zero_centered_gamma;
  a.eps = epsilon;
  a.x_out = x_out;
  a.out = out;
  a.mu = mu;
  a.rsigma = rsigma;
  a.post_mu = post_mu;
  a.post_rsigma = post_rsigma;
  const cudaStream_t s = as_stream(stream);
  if (out_dtype != TE_E4M3 || q->mode == TE_SCALING_DELAYED) {
    a.cast.out_dtype = out_dtype;
    if (out_dtype == TE_E4M3) {
      a.cast.scale = q->scale;
      a.cast.scale_inv_out = q->scale_inv;
    }
    a.cast.amax_out = q ? q->amax : nullptr;
    if (a.cast.amax_out) {
      const te_status st = launch_zero_scalar(a.cast.amax_out, s);
      if (st != TE_OK) return st;
      a.beside_zero = 1;
    }
    return launch_residual_norm_fwd(a, s);
  }
  return run_cast(q, out_dtype, 0, s, [&](const CastSpec& c) {
    a.cast = c;
    return launch_residual_norm_fwd(a, s);
  });
}

size_t te_residual_norm_bwd_workspace(int64_t M, int64_t H, int64_t gates) {
  return residual_norm_bwd_workspace(M, H, gates);
}

te_status te_residual_norm_bwd(const void* dout, const void* dx_out, const void* x_out, const void* y, te_dtype dtype,
                               te_dtype residual_dtype, int64_t M, int64_t H, const float* mu, const float* rsigma,
                               const float* post_mu, const float* post_rsigma, const void* gamma,
                               const void* post_gamma, const void* post_beta, const void* gate, int64_t gates,
                               float residual_scale, te_norm_type norm_type, int zero_centered_gamma, void* dresidual,
                               void* dy, float* dgamma, float* dbeta, float* dpost_gamma, float* dpost_beta,
                               float* dgate, void* workspace, size_t ws_bytes, void* stream) {
  if (M < 0 || H <= 0 || !valid_stream(dtype, residual_dtype) || !valid_norm(norm_type)) return TE_ERR_INVALID_ARG;
  const bool ln = norm_type == TE_LAYERNORM, post = post_gamma != nullptr;
  const int64_t gate_rows = gate_rows_of(gate, gates, M);
  if (gate_rows == 0 || !gamma || !dgamma || (!gate && dgate) ||
      (!post && (post_beta || post_mu || post_rsigma || dpost_gamma || dpost_beta)))
    return TE_ERR_INVALID_ARG;
  if (M > 0 && (!dout || !x_out || !rsigma || (ln && !mu) || ((post || gate) && !y) || (post && !post_rsigma) ||
                (post && ln && !post_mu)))
    return TE_ERR_INVALID_ARG;
  // what is not read may be anything, and lie anywhere
  if (!post && !gate) y = nullptr;
  if (!ln) mu = post_mu = nullptr;
  if (!ln || !dgate) post_beta = nullptr;
  if (H % 8 || H > 8192 || M > kMaxDim) return TE_ERR_UNSUPPORTED;
  for (const void* p : {dout, dx_out, x_out, y, gamma, post_gamma, post_beta, gate, static_cast<const void*>(dresidual),
                        static_cast<const void*>(dy), static_cast<const void*>(workspace)})
    if (!aligned16(p)) return TE_ERR_UNSUPPORTED;
  for (const float* p : {mu, rsigma, post_mu, post_rsigma, static_cast<const float*>(dgamma),
                         static_cast<const float*>(dbeta), static_cast<const float*>(dpost_gamma),
                         static_cast<const float*>(dpost_beta), static_cast<const float*>(dgate)})
    if (!aligned4(p)) return TE_ERR_UNSUPPORTED;
  const cudaStream_t s = as_stream(stream);
  const size_t col = size_t(H) * 4, ngates = gate ? size_t(gates) : 1;
  if (M > 0) {
    const size_t e = esize(dtype), re = esize(residual_dtype), rows = size_t(M) * H, vec = size_t(H) * e;
    const size_t need = residual_norm_bwd_workspace(M, H, gate ? gates : 1);
    if (!workspace || ws_bytes < need) return TE_ERR_WORKSPACE;
    Spans spans;
    spans.reads(dout, rows * e);
    if (dx_out != dresidual) spans.reads(dx_out, rows * re);
    spans.reads(x_out, rows * re);
    spans.reads(y, rows * e);
    for (const float* p : {mu, rsigma, post_mu, post_rsigma}) spans.reads(p, size_t(M) * 4);
    for (const void* p : {gamma, post_gamma, post_beta}) spans.reads(p, vec);
    spans.reads(gate, vec * ngates);
    spans.writes(dresidual, rows * re);
    spans.writes(dy, rows * e);
    for (float* p : {dgamma, dbeta, dpost_gamma, dpost_beta}) spans.writes(p, col);
    spans.writes(dgate, col * ngates);
    spans.writes(workspace, need);
    if (spans.clash()) return TE_ERR_INVALID_ARG;
  }
  // RMSNorm has no shift: the gradient of one is zero, as every gradient is without rows
  te_status st = TE_OK;
  if (M == 0) {
    for (float* p : {dgamma, dpost_gamma})
      if (st == TE_OK) st = zero(p, col, s);
    if (st == TE_OK) st = zero(dgate, col * ngates, s);
  }
  if (!ln || M == 0)
    for (float* p : {dbeta, dpost_beta})
      if (st == TE_OK) st = zero(p, col, s);
  if (st != TE_OK || M == 0) return st;
  ResidualNormBwdArgs a;
  a.dout = dout;
  a.dx_out = dx_out;
  a.x_out = x_out;
  a.y = y;
  a.dtype = dtype;
  a.residual_dtype = residual_dtype;
  a.M = M;
  a.H = H;
  a.mu = mu;
  a.rsigma = rsigma;
  a.post_mu = post_mu;
  a.post_rsigma = post_rsigma;
  a.gamma = gamma;
  a.post_gamma = post_gamma;
  a.post_beta = post_beta;
  a.gate = gate;
  a.gate_rows = gate_rows;
  a.residual_scale = residual_scale;
  a.norm_type = norm_type;
  a.zero_centered_gamma = zero_centered_gamma;
  a.dresidual = dresidual;
  a.dy = dy;
  a.dgamma = dgamma;
  a.dbeta = ln ? dbeta : nullptr;
  a.dpost_gamma = dpost_gamma;
  a.dpost_beta = ln ? dpost_beta : nullptr;
  a.dgate = dgate;
  a.partials = static_cast<float*>(workspace);
  return launch_residual_norm_bwd(a, s);
}

size_t te_dense_residual_fwd_workspace(int64_t M, int64_t K, int64_t N, te_dtype dtype) {
  return dense_fwd_workspace(M, K, N, dtype);
}

te_status te_dense_residual_fwd(const void* x, const void* kernel, te_dtype dtype, const float* x_scale_inv,
                                const float* kernel_scale_inv, const void* bias, te_act_type act, const void* gate,
                                int64_t gates, const void* residual, te_dtype residual_dtype, float residual_scale,
                                int64_t M, int64_t K, int64_t N, void* out, void* saved_z, void* workspace,
                                size_t ws_bytes, void* stream) {
  if (M < 0 || K <= 0 || N <= 0 || (dtype != TE_BF16 && dtype != TE_E4M3) || !is_act_dtype(residual_dtype) ||
      act < TE_IDENTITY || act > TE_SILU || (dtype == TE_BF16 && (x_scale_inv || kernel_scale_inv)))
    return TE_ERR_INVALID_ARG;
  if (M > 0 && (!x || !kernel || !residual || !out)) return TE_ERR_INVALID_ARG;
  const int64_t gate_rows = gate_rows_of(gate, gates, M);
  if (gate_rows == 0) return TE_ERR_INVALID_ARG;
  if (K % 16 || N % 16 || M > kMaxDim || K > kMaxDim || N > kMaxDim) return TE_ERR_UNSUPPORTED;
  for (const void* p : {x, kernel, bias, gate, residual, static_cast<const void*>(out),
                        static_cast<const void*>(saved_z), static_cast<const void*>(workspace)})
    if (!aligned16(p)) return TE_ERR_UNSUPPORTED;
  if (!aligned4(x_scale_inv) || !aligned4(kernel_scale_inv)) return TE_ERR_UNSUPPORTED;
  if (M == 0) return TE_OK;
  const size_t e = esize(dtype), re = esize(residual_dtype), rows = size_t(M) * N;
  const size_t used = workspace ? std::min(ws_bytes, dense_fwd_workspace(M, K, N, dtype)) : 0;
  Spans spans;
  spans.reads(x, size_t(M) * K * e);
  spans.reads(kernel, size_t(K) * N * e);
  spans.reads(x_scale_inv, 4);
  spans.reads(kernel_scale_inv, 4);
  spans.reads(bias, size_t(N) * 2);
  spans.reads(gate, gate ? size_t(N) * 2 * size_t(gates) : 0);
  if (out != residual) spans.reads(residual, rows * re);
  spans.writes(out, rows * re);
  spans.writes(saved_z, rows * 2);
  spans.writes(workspace, used);
  if (spans.clash()) return TE_ERR_INVALID_ARG;
  GemmArgs g;
  g.A = x;
  g.B = kernel;
  g.ab_dtype = dtype;
  g.a_kmajor = 1;
  g.b_kmajor = 0;
  g.M = M;
  g.N = N;
  g.K = K;
  g.a_scale_inv = x_scale_inv;
  g.b_scale_inv = kernel_scale_inv;
  g.epilogue = EPI_RESIDUAL;
  g.act = act;
  g.bias = bias;
  g.bias_dtype = TE_BF16;
  g.saved_h = saved_z;
  g.residual = residual;
  g.residual_scale = residual_scale;
  g.gate = gate;
  g.gate_rows = gate_rows;
  g.D = out;
  g.cast.out_dtype = residual_dtype;
  g.split_ws = workspace;
  g.split_ws_bytes = used;
  return dense_few_serves(M, N, K, dtype) ? launch_dense_few(g, as_stream(stream)) : launch_gemm(g, as_stream(stream));
}

size_t te_dense_residual_bwd_workspace(int64_t M, int64_t K, int64_t N, int64_t gates, te_dtype dtype) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  return dense_bwd_layout(nullptr, M, K, N, gates, dtype).bytes;
}

te_status te_dense_residual_bwd(const void* dout, te_dtype residual_dtype, const void* x, const void* kernel,
                                te_dtype dtype, const void* saved_z, te_act_type act, const void* gate, int64_t gates,
                                float residual_scale, const te_quantizer* q, const float* x_scale_inv,
                                const float* kernel_scale_inv, int64_t M, int64_t K, int64_t N, void* dx, void* dkernel,
                                void* dresidual, float* dbias, float* dgate, void* workspace, size_t ws_bytes,
                                void* stream) {
  if (M < 0 || K <= 0 || N <= 0 || (dtype != TE_BF16 && dtype != TE_E4M3) || !is_act_dtype(residual_dtype) ||
      act < TE_IDENTITY || act > TE_SILU)
    return TE_ERR_INVALID_ARG;
  const bool quant = dtype == TE_E4M3;
  if (quant ? (!enabled(q) || !quantizer_ok(q) || !q->scale_inv) : (q || x_scale_inv || kernel_scale_inv))
    return TE_ERR_INVALID_ARG;
  const int64_t gate_rows = gate_rows_of(gate, gates, M);
  if (gate_rows == 0 || (!gate && dgate) || !dkernel) return TE_ERR_INVALID_ARG;
  if (M > 0 && (!dout || !x || !kernel || !dx || ((act != TE_IDENTITY || dgate) && !saved_z)))
    return TE_ERR_INVALID_ARG;
  if (act == TE_IDENTITY && !dgate) saved_z = nullptr;  // not read
  if (K % 16 || N % 16 || M > kMaxDim || K > kMaxDim || N > kMaxDim) return TE_ERR_UNSUPPORTED;
  for (const void* p : {dout, x, kernel, saved_z, gate, static_cast<const void*>(dx), static_cast<const void*>(dkernel),
                        static_cast<const void*>(dresidual), static_cast<const void*>(workspace)})
    if (!aligned16(p)) return TE_ERR_UNSUPPORTED;
  for (const float* p : {x_scale_inv, kernel_scale_inv, static_cast<const float*>(dbias), static_cast<const float*>(dgate)})
    if (!aligned4(p)) return TE_ERR_UNSUPPORTED;
  const cudaStream_t s = as_stream(stream);
  const size_t ngates = gate ? size_t(gates) : 1;
  te_status st = TE_OK;
  if (M == 0) {
    st = zero(dkernel, size_t(K) * N * 2, s);
    if (st == TE_OK) st = zero(dbias, size_t(N) * 4, s);
    return st == TE_OK ? zero(dgate, size_t(N) * 4 * ngates, s) : st;
  }
  const DenseBwdLayout L = dense_bwd_layout(workspace, M, K, N, int64_t(ngates), dtype);
  if (!workspace || ws_bytes < L.split.required) return TE_ERR_WORKSPACE;
  const size_t e = esize(dtype), re = esize(residual_dtype), rows = size_t(M) * N;
  Spans spans;
  spans.reads(x, size_t(M) * K * e);
  spans.reads(kernel, size_t(K) * N * e);
  spans.reads(x_scale_inv, 4);
  spans.reads(kernel_scale_inv, 4);
  spans.reads(saved_z, rows * 2);
  spans.reads(gate, gate ? size_t(N) * 2 * ngates : 0);
  spans.reads(dout, rows * re);
  spans.writes(dx, size_t(M) * K * 2);
  spans.writes(dkernel, size_t(K) * N * 2);
  spans.writes(dresidual, rows * re);
  spans.writes(dbias, size_t(N) * 4);
  spans.writes(dgate, size_t(N) * 4 * ngates);
  spans.writes(workspace, std::min(ws_bytes, L.bytes));
  spans.quantizer(q);
  if (spans.clash()) return TE_ERR_INVALID_ARG;
  // a bf16 dout without a gate or an activation is dz itself
  const bool same = !quant && residual_dtype == TE_BF16 && act == TE_IDENTITY && !gate;
  if (!same || dbias || dresidual) {
    DenseResidualGradArgs a;
    a.dout = dout;
    a.z = saved_z;
    a.dtype = residual_dtype;
    a.M = M;
    a.N = N;
    a.act = act;
    a.gate = gate;
    a.gate_rows = gate_rows;
    a.residual_scale = residual_scale;
    a.partials = L.partials;
    a.dz = same ? nullptr : L.dz;
    // with current scaling the sums and dresidual come from the amax pass, the cast pass only stores dz
    const bool two_pass = quant && q->mode == TE_SCALING_CURRENT;
    st = run_cast(quant ? q : nullptr, quant ? int(TE_E4M3) : int(TE_BF16), 0, s, [&](const CastSpec& c) {
      const bool here = !two_pass || c.store == 0;
      a.dresidual = here ? dresidual : nullptr;
      a.dbias = here ? dbias : nullptr;
      a.dgate = here ? dgate : nullptr;
      a.cast = c;
      return launch_dense_residual_grad(a, s);
    });
    if (st != TE_OK) return st;
  }
  const void* dz = same ? dout : L.dz;
  GemmArgs g;  // dx = dz kernel^T, the contraction over N
  g.A = dz;
  g.B = kernel;
  g.ab_dtype = dtype;
  g.a_kmajor = 1;
  g.b_kmajor = 1;
  g.M = M;
  g.N = K;
  g.K = N;
  g.a_scale_inv = quant ? q->scale_inv : nullptr;
  g.b_scale_inv = kernel_scale_inv;
  g.D = dx;
  g.cast.out_dtype = TE_BF16;
  give_split(g, L.split, workspace, ws_bytes);
  g.order = PRODUCT_BEFORE;
  // (Few tiles of one row: above 128 rows the tiles of launch_gemm leave SMs on which the second product starts.
  // Both products and the gradient in front, us, few tiles / those: 4096 x 4096 in bf16 at one row 38 / 57, at 128
  // 44 / 59, at 512 58 / 58; 1024 x 1024 at 128 15 / 18, at 512 24 / 20.)
  st = M <= 128 && dense_few_serves(M, K, N, dtype) ? launch_dense_few(g, s) : launch_gemm(g, s);
  if (st != TE_OK) return st;
  GemmArgs h;  // dkernel = x^T dz, the contraction over the rows
  h.A = x;
  h.B = dz;
  h.ab_dtype = dtype;
  h.a_kmajor = 0;
  h.b_kmajor = 0;
  h.M = K;
  h.N = N;
  h.K = M;
  h.a_scale_inv = x_scale_inv;
  h.b_scale_inv = quant ? q->scale_inv : nullptr;
  h.D = dkernel;
  h.cast.out_dtype = TE_BF16;
  give_split(h, L.split, workspace, ws_bytes);
  h.order = PRODUCT_BESIDE;
  return launch_gemm(h, s);
}

size_t te_grad_norm_workspace(int64_t n) { return grad_norm_workspace(n); }

te_status te_grad_norm(const te_grad* g, int64_t n, float* norm, void* workspace, size_t ws_bytes, void* stream) {
  return grads(g, n, false, 0.0, 0.0, norm, workspace, ws_bytes, as_stream(stream));
}

te_status te_clip_grad_norm(const te_grad* g, int64_t n, double max_norm, double epsilon, float* norm, void* workspace,
                            size_t ws_bytes, void* stream) {
  if (!(max_norm >= 0.0) || !std::isfinite(max_norm) || !(epsilon >= 0.0) || !std::isfinite(epsilon))
    return TE_ERR_INVALID_ARG;
  return grads(g, n, true, max_norm, epsilon, norm, workspace, ws_bytes, as_stream(stream));
}

}  // extern "C"

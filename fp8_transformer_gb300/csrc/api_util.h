// Argument checks, workspace carving and the cast passes shared by the C entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "kernels.h"
#include "te_gb300.h"

namespace te {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool opt_aligned16(const void* p) { return p == nullptr || aligned16(p); }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline size_t esize(int dt) { return dt == TE_F32 ? 4 : dt == TE_BF16 ? 2 : 1; }
inline bool is_act_dtype(int dt) { return dt == TE_F32 || dt == TE_BF16; }
inline bool valid_act(int a) { return a >= TE_IDENTITY && a <= TE_REGLU; }
inline bool enabled(const te_quantizer* q) { return q != nullptr && q->scale != nullptr; }

inline bool quantizer_ok(const te_quantizer* q) {
  if (!enabled(q)) return true;
  if (!aligned4(q->scale) || !aligned4(q->scale_inv) || !aligned4(q->amax)) return false;
  if (q->mode != TE_SCALING_DELAYED && q->mode != TE_SCALING_CURRENT) return false;
  // Current scaling keeps this call's amax between its two passes.
  if (q->mode == TE_SCALING_CURRENT && q->amax == nullptr) return false;
  return true;
}

constexpr size_t kAlign = 256;
inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Sequential carving of the caller's workspace into 256-byte aligned regions.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  explicit Carver(void* b) : base(static_cast<uint8_t*>(b)) {}
  void* take(size_t bytes) {
    void* p = base ? base + used : nullptr;
    used += round_up(bytes);
    return p;
  }
};

// The scratch for splitting GEMM tails along K (launch_gemm) is carved last: a workspace that
// stops short of it still serves the call, with no tile split.  The GEMMs of one call run one
// after another on its stream, so they share the region, sized for the largest.
struct SplitScratch {
  size_t offset = 0;  // where the region starts in the workspace
  size_t required = 0;  // workspace bytes the call needs (everything before the region)
};

inline SplitScratch carve_split(Carver& c, std::initializer_list<size_t> needs) {
  SplitScratch r;
  r.required = c.used;
  r.offset = c.used;
  size_t most = 0;
  for (size_t n : needs) most = n > most ? n : most;
  if (most) c.take(most);
  return r;
}

inline void give_split(GemmArgs& g, const SplitScratch& sc, void* ws, size_t ws_bytes) {
  if (ws && ws_bytes > sc.offset) {
    g.split_ws = static_cast<uint8_t*>(ws) + sc.offset;
    g.split_ws_bytes = ws_bytes - sc.offset;
  }
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

inline te_status zero_scalar(float* p, cudaStream_t s) {
  if (!p) return TE_OK;
  return cudaMemsetAsync(p, 0, sizeof(float), s) == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

// Runs a bandwidth-bound producer once (no quantizer, or delayed scaling) or twice (current
// scaling: an amax pass that stores nothing, then the cast pass with scale = 448 / amax).
template <class Launch>
te_status run_cast(const te_quantizer* q, int out_dtype, int fake_quant, cudaStream_t s,
                   Launch&& launch) {
  CastSpec c;
  c.out_dtype = out_dtype;
  c.fake_quant = fake_quant;
  if (q) {
    te_status st = zero_scalar(q->amax, s);
    if (st != TE_OK) return st;
  }
  if (!enabled(q)) {
    c.amax_out = q ? q->amax : nullptr;
    return launch(c);
  }
  if (q->mode == TE_SCALING_DELAYED) {
    c.scale = q->scale;
    c.amax_out = q->amax;
    c.scale_inv_out = q->scale_inv;
    return launch(c);
  }
  CastSpec pass1 = c;
  pass1.store = 0;
  pass1.amax_out = q->amax;
  te_status st = launch(pass1);
  if (st != TE_OK) return st;
  CastSpec pass2 = c;
  pass2.amax_in = q->amax;
  pass2.scale_out = q->scale;
  pass2.scale_inv_out = q->scale_inv;
  return launch(pass2);
}

// The gradient from a checkpoint with its cast.  Current scaling: dbias and act_out come from the
// amax pass, the cast pass only stores dx.
inline te_status dact_ckpt_cast(DactCkptArgs a, const te_quantizer* q, int dx_dtype, void* act_out,
                                float* dbias, cudaStream_t s) {
  const bool two_pass = enabled(q) && q->mode == TE_SCALING_CURRENT;
  return run_cast(q, dx_dtype, 0, s, [&](const CastSpec& c) {
    const bool here = two_pass ? c.store == 0 : true;
    a.act_out = here ? act_out : nullptr;
    a.dbias = here ? dbias : nullptr;
    a.cast = c;
    return launch_dact_ckpt(a, s);
  });
}

}  // namespace te

// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <utility>

#include "te_gb300.h"

namespace te {

// Gated activations take [gate | linear] and apply their base function to the gate half.
__host__ __device__ constexpr bool is_gated(int act) {
  return act == TE_SWIGLU || act == TE_GEGLU || act == TE_REGLU;
}
__host__ __device__ constexpr int gate_act(int act) {
  return act == TE_SWIGLU ? TE_SILU : act == TE_GEGLU ? TE_GELU : act == TE_REGLU ? TE_RELU : act;
}

// Output stage shared by the bandwidth-bound kernels: how fp32 results become the stored
// tensor, and which scalars the kernel reads or writes.
struct CastSpec {
  int out_dtype = TE_BF16;         // TE_F32 / TE_BF16 / TE_E4M3
  int fake_quant = 0;              // quantize then dequantize into out_dtype (F32 / BF16)
  const float* scale = nullptr;    // E4M3 scale to use (delayed scaling)
  const float* amax_in = nullptr;  // current scaling: derive the scale from this amax
  float* amax_out = nullptr;       // atomic max of |pre-cast value| (zeroed by the caller)
  float* scale_out = nullptr;      // written with the scale used (current scaling)
  float* scale_inv_out = nullptr;  // written with 1 / scale
  int store = 1;                   // 0: amax pass of current scaling, nothing stored
};

struct NormFwdArgs {
  const void* x = nullptr;
  int x_dtype = TE_BF16;
  int64_t M = 0, H = 0;
  const void* gamma = nullptr;
  const void* beta = nullptr;
  int norm_type = TE_LAYERNORM;
  int zero_centered_gamma = 0;
  float eps = 1e-6f;
  void* out = nullptr;
  float* mu = nullptr;
  float* rsigma = nullptr;
  CastSpec cast;
  int prefetch = 0;  // rows ahead of the current one each warp asks L2 to fetch (set at launch)
};
te_status launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s);

struct NormBwdArgs {
  const void* dz = nullptr;  // [M, H] upstream gradient, dtype
  const void* x = nullptr;   // [M, H] forward input, dtype
  const float* mu = nullptr;
  const float* rsigma = nullptr;
  const void* gamma = nullptr;
  int dtype = TE_BF16;
  int64_t M = 0, H = 0;
  int norm_type = TE_LAYERNORM;
  int zero_centered_gamma = 0;
  void* dx = nullptr;        // [M, H] dtype
  float* dgamma = nullptr;   // [H]
  float* dbeta = nullptr;    // [H] or null
  float* partials = nullptr; // workspace: [chunks, 2, H]
};
te_status launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s);

// p = norm(y) or y, x_out = residual_scale * residual + gate * p, out = norm(x_out).
struct ResidualNormArgs {
  const void* y = nullptr;         // [M, H] y_dtype
  const void* residual = nullptr;  // [M, H] residual_dtype
  int y_dtype = TE_BF16, residual_dtype = TE_BF16;
  int64_t M = 0, H = 0;
  const void* gamma = nullptr;       // [H] y_dtype, like the vectors below
  const void* beta = nullptr;
  const void* post_gamma = nullptr;  // null: no norm of y
  const void* post_beta = nullptr;
  const void* gate = nullptr;        // [M / gate_rows, H] or null
  int64_t gate_rows = 1;             // rows that share a gate row
  float residual_scale = 1.0f;
  int norm_type = TE_LAYERNORM;
  int zero_centered_gamma = 0;
  float eps = 1e-6f;
  void* x_out = nullptr;  // [M, H] residual_dtype; may be residual
  void* out = nullptr;
  float* mu = nullptr;
  float* rsigma = nullptr;
  float* post_mu = nullptr;
  float* post_rsigma = nullptr;
  CastSpec cast;
  // the kernel in front on the stream only zeroes cast.amax_out: start beside it, wait before the amax
  int beside_zero = 0;
};
// *p = 0, by a kernel beside which a dependent may start.
te_status launch_zero_scalar(float* p, cudaStream_t s);
te_status launch_residual_norm_fwd(const ResidualNormArgs& a, cudaStream_t s);

struct ResidualNormBwdArgs {
  const void* dout = nullptr;    // [M, H] dtype
  const void* dx_out = nullptr;  // [M, H] residual_dtype, or null
  const void* x_out = nullptr;   // [M, H] residual_dtype
  const void* y = nullptr;       // [M, H] dtype; read with a post norm or a gate
  int dtype = TE_BF16, residual_dtype = TE_BF16;
  int64_t M = 0, H = 0;
  const float* mu = nullptr;
  const float* rsigma = nullptr;
  const float* post_mu = nullptr;
  const float* post_rsigma = nullptr;
  const void* gamma = nullptr;
  const void* post_gamma = nullptr;
  const void* post_beta = nullptr;
  const void* gate = nullptr;
  int64_t gate_rows = 1;
  float residual_scale = 1.0f;
  int norm_type = TE_LAYERNORM;
  int zero_centered_gamma = 0;
  void* dresidual = nullptr;  // [M, H] residual_dtype or null; may be dx_out
  void* dy = nullptr;         // [M, H] dtype or null
  float* dgamma = nullptr;
  float* dbeta = nullptr;
  float* dpost_gamma = nullptr;
  float* dpost_beta = nullptr;
  float* dgate = nullptr;          // [M / gate_rows, H]
  float* partials = nullptr;       // workspace
  float* gate_partials = nullptr;  // set at launch, like rows_per_cta
  int64_t rows_per_cta = 1;
};
te_status launch_residual_norm_bwd(const ResidualNormBwdArgs& a, cudaStream_t s);
size_t residual_norm_bwd_workspace(int64_t M, int64_t H, int64_t gates);

// Workspace of te_layernorm_mlp_fwd_host: device staging of x and out plus one forward's.
size_t host_fwd_workspace(int64_t M, int64_t H, int64_t F, int dtype, int act);
size_t norm_bwd_workspace(int64_t M, int64_t H);
// Workspaces of the 4-bit dense layer, for either format.
size_t dense_fp4_fwd_workspace(int64_t M, int64_t K);
size_t dense_fp4_bwd_workspace(int64_t M, int64_t N);

struct ActArgs {
  const void* x = nullptr;
  int x_dtype = TE_BF16;
  int64_t M = 0, N_in = 0;
  int act = TE_GELU;
  void* out = nullptr;
  CastSpec cast;
};
te_status launch_act_lu(const ActArgs& a, cudaStream_t s);

struct DactArgs {
  const void* dy = nullptr;
  const void* x = nullptr;
  int dtype = TE_BF16;
  int64_t M = 0, N_in = 0;
  int act = TE_GELU;
  void* dx = nullptr;
  float* dbias = nullptr;
  float* partials = nullptr;  // workspace for the deterministic column reduction
  CastSpec cast;
};
te_status launch_dact_dbias(const DactArgs& a, cudaStream_t s);
size_t dact_dbias_workspace(int64_t M, int64_t N_in);

// The same from an 8-bit checkpoint of the activation's input, which also gives back act(h).
struct DactCkptArgs {
  const void* dy = nullptr;      // [M, n_out]
  const void* codes = nullptr;   // [M, N_in] E4M3, MXFP8
  const void* scales = nullptr;
  int dtype = TE_BF16;
  int64_t M = 0, N_in = 0;
  int act = TE_GELU;
  void* dx = nullptr;            // [M, N_in]
  void* act_out = nullptr;       // [M, n_out] act(h) in dtype, or null
  float* dbias = nullptr;
  float* partials = nullptr;     // as for DactArgs
  CastSpec cast;
};
te_status launch_dact_ckpt(const DactCkptArgs& a, cudaStream_t s);

struct QuantizeArgs {
  const void* x = nullptr;
  int x_dtype = TE_BF16;
  int64_t n = 0;  // elements, multiple of 8
  void* out = nullptr;
  CastSpec cast;
};
te_status launch_quantize(const QuantizeArgs& a, cudaStream_t s);

// Block-scaled formats (te_block_format): elements in a block, and codes per byte.
__host__ __device__ constexpr int block_len(int fmt) { return fmt == TE_NVFP4 ? 16 : 32; }
__host__ __device__ constexpr int codes_per_byte(int fmt) { return fmt == TE_MXFP8 ? 1 : 2; }
// Scale tiles along one row of tiles, and the bytes of a [rows, cols] tensor's scales.
__host__ __device__ constexpr int64_t scale_groups(int fmt, int64_t cols) {
  return (cols / block_len(fmt) + 3) / 4;
}
inline size_t block_scale_bytes(int fmt, int64_t rows, int64_t cols) {
  return size_t((rows + 127) / 128) * size_t(scale_groups(fmt, cols)) * 512;
}
// Length of a packed transposed row: the rows of x in whole blocks of 32.
inline int64_t pad32(int64_t n) { return (n + 31) / 32 * 32; }

struct BlockQuantArgs {
  const void* x = nullptr;  // [M, N]
  int x_dtype = TE_BF16;
  int64_t M = 0, N = 0;     // N a multiple of 32 (16 without codes)
  int fmt = TE_MXFP4;
  void* codes = nullptr;    // [M, N] packed along N, or null
  void* scales = nullptr;
  void* codes_t = nullptr;  // [N, pad32(M)] packed along M, or null
  int64_t pitch_t = 0;      // bytes from one row of codes_t to the next (0: none between them)
  void* scales_t = nullptr;
  const float* scale = nullptr;    // NVFP4: the tensor scale given (delayed scaling)
  const float* amax_in = nullptr;  // NVFP4: derive the tensor scale from this amax
  float* amax_out = nullptr;       // atomic max of |x| (zeroed by the caller)
  float* scale_out = nullptr;      // written with the tensor scale used
  float* scale_inv_out = nullptr;  // written with 1 / scale
  float* partials = nullptr;       // column sums of each 128-row tile [ceil(M / 128), N], or null
};
te_status launch_block_quantize(const BlockQuantArgs& a, cudaStream_t s);
// amax_out = max |x| of n elements (a multiple of 8), zeroed first.
te_status launch_amax(const void* x, int x_dtype, int64_t n, float* amax_out, cudaStream_t s);
// out[j] = sum over the chunks of partials[c][j], in a fixed order (n a multiple of 4); launched
// as a programmatic dependent of the kernel that wrote the partials.
te_status launch_colsum(const float* partials, int chunks, int64_t n, float* out, cudaStream_t s);

struct BlockDequantArgs {
  const void* codes = nullptr;
  const void* scales = nullptr;
  int fmt = TE_MXFP4;
  const float* scale_inv = nullptr;  // NVFP4: the tensor's factor, or null (= 1)
  int64_t M = 0, N = 0;
  void* out = nullptr;
  int out_dtype = TE_BF16;
};
te_status launch_block_dequantize(const BlockDequantArgs& a, cudaStream_t s);

// dst[C, R] = transpose of src[R, C] (fp32): the tf32 tensor-core path takes K-major operands.
te_status launch_transpose_f32(const float* src, int64_t R, int64_t C, float* dst, cudaStream_t s);

// scale = 448 / amax (the recipe's exceptions included), scale_inv = 1 / scale, for up to
// kMaxScaleUpdates quantizers in one launch.
constexpr int kMaxScaleUpdates = 16;
struct ScaleUpdateArgs {
  int n = 0;
  const float* amax[kMaxScaleUpdates] = {};
  float* scale[kMaxScaleUpdates] = {};
  float* scale_inv[kMaxScaleUpdates] = {};
};
te_status launch_update_scales(const ScaleUpdateArgs& a, cudaStream_t s);

// Tensor-core GEMM D[M, N] = epilogue(alpha * op(A) op(B)).
// EPI_RESIDUAL: D = residual_scale * residual + gate * act(alpha op(A) op(B) + bias); A K-major, B
// stored [K, N], bf16 or E4M3.
enum Epilogue { EPI_BIAS = 0, EPI_BIAS_ACT = 1, EPI_BIAS_GATED = 2, EPI_RESIDUAL = 3 };

// Two products in a row of which the second reads nothing that the first writes.  (Neither may write what the
// other reads or writes; a second product that splits along K clears its flags behind the first and waits.)
enum GemmOrder {
  PRODUCT_ALONE = 0,
  PRODUCT_BEFORE = 1,  // the first: lets the second in
  PRODUCT_BESIDE = 2,  // the second: starts while the first ends
};

struct GemmArgs {
  const void* A = nullptr;
  const void* B = nullptr;
  int ab_dtype = TE_BF16;   // TE_BF16 / TE_E4M3 / TE_F32 (tf32)
  int a_kmajor = 1;         // A stored [M, K] (1) or [K, M] (0)
  int b_kmajor = 0;         // B stored [N, K] (1) or [K, N] (0)
  int64_t M = 0, N = 0, K = 0;  // N = accumulator columns; gated: N = 2F
  const float* a_scale_inv = nullptr;
  const float* b_scale_inv = nullptr;
  int epilogue = EPI_BIAS;
  int act = TE_IDENTITY;
  const void* bias = nullptr;   // [N]
  int bias_dtype = TE_F32;
  int h_dtype = TE_F32;         // dtype the pre-activation is rounded to (act epilogues)
  void* saved_h = nullptr;      // [M, N] pre-activation, h_dtype
  void* h_codes = nullptr;      // [M, N] pre-activation in MXFP8 (N a multiple of 32), or null
  void* h_scales = nullptr;
  const void* residual = nullptr;  // EPI_RESIDUAL: [M, N] in D's dtype; may be D
  float residual_scale = 1.0f;
  const void* gate = nullptr;      // [M / gate_rows, N] bf16, or null
  int64_t gate_rows = 1;
  void* D = nullptr;            // [M, N] or [M, N/2] gated
  CastSpec cast;                // output stage of D (amax / E4M3 of the activation)
  // Optional scratch (256-byte aligned) for splitting the last wave's tiles along K; without it
  // no tile is split.
  void* split_ws = nullptr;
  size_t split_ws_bytes = 0;
  int order = PRODUCT_ALONE;
};
te_status launch_gemm(const GemmArgs& g, cudaStream_t s);
// Bytes of split_ws that launch_gemm would use for this GEMM on the current device (0: none).
size_t gemm_split_workspace(int64_t M, int64_t N, int64_t K, int ab_dtype, int epilogue);

// EPI_RESIDUAL with B stored [K, N], or EPI_BIAS without a bias with B stored [N, K], for outputs of few tiles, split
// along K over a cluster; and whether it is the faster way.
bool dense_few_serves(int64_t M, int64_t N, int64_t K, int ab_dtype);
te_status launch_dense_few(const GemmArgs& g, cudaStream_t s);

// Product of two packed 4-bit operands: D[M, N] = alpha * A B^T + bias, A [M, K], B [N, K].
struct BlockGemmArgs {
  const void* A = nullptr;         // codes, K / 2 bytes a row
  const void* a_scales = nullptr;
  const void* B = nullptr;
  const void* b_scales = nullptr;
  int fmt = TE_MXFP4;
  int64_t M = 0, N = 0, K = 0;     // K a multiple of 32, N of 16
  int64_t b_pitch = 0;             // bytes from one row of B to the next, a multiple of 16 (0: K / 2)
  const float* a_scale_inv = nullptr;
  const float* b_scale_inv = nullptr;
  const void* bias = nullptr;      // [N]
  int bias_dtype = TE_F32;
  void* D = nullptr;               // [M, N]
  int d_dtype = TE_BF16;
  // B and its scales were complete before the kernel that precedes this one on the stream began,
  // so that their loads may start before that kernel has finished.
  int b_ready = 0;
};
te_status launch_block_gemm(const BlockGemmArgs& a, cudaStream_t s);
// The product with its A operand packed inside the kernel: x is q.x [M, K] with q's tensor scale
// (q.codes and the other outputs unused), g.A, g.a_scales and g.a_scale_inv unset.  For rows up to
// kFewPacked only (TE_ERR_UNSUPPORTED beyond).
constexpr int64_t kFewPacked = 8;
te_status launch_block_gemm_packing(const BlockGemmArgs& g, const BlockQuantArgs& q, cudaStream_t s);

// The gradient of that epilogue: dz = gate * dout * act'(z), with its column sums (dbias), those of
// dout * act(z) over each gate's rows (dgate), and residual_scale * dout.
struct DenseResidualGradArgs {
  const void* dout = nullptr;  // [M, N] dtype
  const void* z = nullptr;     // [M, N] bf16; read with an activation or for dgate
  int dtype = TE_BF16;
  int64_t M = 0, N = 0;
  int act = TE_IDENTITY;
  const void* gate = nullptr;  // [M / gate_rows, N] bf16, or null
  int64_t gate_rows = 1;
  float residual_scale = 1.0f;
  void* dz = nullptr;          // [M, N] bf16 or E4M3, or null
  void* dresidual = nullptr;   // [M, N] dtype, or null
  float* dbias = nullptr;
  float* dgate = nullptr;      // [M / gate_rows, N]
  float* partials = nullptr;   // workspace
  int64_t chunk_rows = 0;      // set at launch, like cols
  int64_t cols = 0;            // of N, those of one launch
  CastSpec cast;
};
te_status launch_dense_residual_grad(DenseResidualGradArgs a, cudaStream_t s);
size_t dense_residual_grad_workspace(int64_t M, int64_t N, int64_t gates);

// Sum of the squares of many tensors, and the tensors scaled by min(1, max_norm / (norm + eps)).
using GradTensor = te_grad;  // `out` set
struct alignas(16) GradSlot {  // a part of the sum: hi + lo + rest
  float hi, lo;
  double rest;
};
// The squares, into slots in the workspace (*used: how many).
te_status launch_grad_squares(const GradTensor* t, int64_t count, GradSlot* slots, int* used, cudaStream_t s);
// norm = the square root of the slots' sum.
te_status launch_grad_norm(const GradSlot* slots, int used, float* norm, cudaStream_t s);
te_status launch_grad_clip(const GradTensor* t, int64_t count, const GradSlot* slots, int used, double max_norm,
                           double eps, float* norm, cudaStream_t s);
size_t grad_norm_workspace(int64_t count);

// Device status word (TE_OK or the first failure a kernel recorded).
int* device_status_ptr();
te_status read_and_clear_device_status(int32_t* out);

int num_sms();

// The streaming reference of te_stream_probe (n_out 16-byte vectors written, each from `ratio`
// read; n_out = 0: n_read vectors read only).
te_status launch_stream_probe(const uint4* src, uint4* dst, size_t n_out, int ratio,
                              size_t n_read, cudaStream_t s);

// Launches `kernel` as a programmatic dependent of the work queued before it on `s`: its launch
// may overlap the previous kernel's tail once every CTA of that kernel has executed
// griddepcontrol.launch_dependents (or exited), and the kernel itself executes
// griddepcontrol.wait before it reads anything the previous kernel wrote.
template <typename... KArgs, typename... Args>
te_status launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s,
                           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess ? TE_OK
                                                                                     : TE_ERR_CUDA;
}

// A value set up once per device and shared by every host thread: get() runs make(&value) for
// the current device the first time (make returns false on failure, and is then retried on the
// next call) and returns the cached value afterwards.  Devices numbered kMaxDevices or above
// are set up on every call, uncached.
constexpr int kMaxDevices = 64;
template <typename T>
class PerDevice {
 public:
  template <class Make>
  bool get(T* out, Make&& make) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 0 || dev >= kMaxDevices) return make(out);
    std::lock_guard<std::mutex> lock(mu_);
    if (!have_[dev]) {
      if (!make(&value_[dev])) return false;
      have_[dev] = true;
    }
    *out = value_[dev];
    return true;
  }

 private:
  std::mutex mu_;
  T value_[kMaxDevices] = {};
  bool have_[kMaxDevices] = {};
};

// 2-D TMA tensor map over a row-major [outer, inner] matrix of dtype, boxes of
// box_inner x box_outer elements, a swizzle of 128 or 64 bytes or none (0), out-of-bounds reads zero.
// pitch: bytes from row to row (0: none between them).
bool make_tmap_2d(CUtensorMap* tm, const void* ptr, int dtype, uint64_t inner, uint64_t outer,
                  uint32_t box_inner, uint32_t box_outer, int swizzle, uint64_t pitch = 0);

// 2-D TMA tensor map over block scales: rows of tiles by 512-byte tiles, boxes of box_rows rows
// of tiles x box_tiles tiles, out-of-bounds reads zero.
bool make_tmap_scales(CUtensorMap* tm, const void* ptr, uint64_t tiles, uint64_t tile_rows,
                      uint32_t box_tiles, uint32_t box_rows);

// Brackets one kernel launch with profiling events when te_profile_begin is active.
class ProfileScope {
 public:
  ProfileScope(int kind, cudaStream_t stream);
  ~ProfileScope();
  ProfileScope(const ProfileScope&) = delete;
  ProfileScope& operator=(const ProfileScope&) = delete;

 private:
  int kind_;
  cudaStream_t stream_;
  int slot_ = -1;
};

}  // namespace te

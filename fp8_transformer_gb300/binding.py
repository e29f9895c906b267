"""ctypes binding of libte_gb300.so (the C ABI declared in include/te_gb300.h).

Argument marshalling only: each function takes torch tensors, checks their dtype/shape against
the C signature, and passes raw device pointers and sizes.  Every step of the computation runs
in the library's CUDA kernels; there is no fallback.  A missing or unbuildable library raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

(TE_OK, TE_ERR_INVALID_ARG, TE_ERR_UNSUPPORTED, TE_ERR_CUDA, TE_ERR_TIMEOUT, TE_ERR_WORKSPACE,
 TE_ERR_TOO_LARGE) = range(7)
TE_F32, TE_BF16, TE_E4M3 = 0, 1, 2
TE_LAYERNORM, TE_RMSNORM = 0, 1
TE_IDENTITY, TE_RELU, TE_GELU, TE_SILU, TE_SWIGLU, TE_GEGLU, TE_REGLU = range(7)
TE_SCALING_DELAYED, TE_SCALING_CURRENT = 0, 1
(TE_OP_NORM_FWD, TE_OP_ACT_LU, TE_OP_DACT_DBIAS, TE_OP_LAYERNORM_DENSE_FWD,
 TE_OP_LAYERNORM_MLP_FWD, TE_OP_NORM_BWD, TE_OP_LAYERNORM_MLP_BWD,
 TE_OP_LAYERNORM_DENSE_BWD, TE_OP_LAYERNORM_MLP_FWD_HOST, TE_OP_GEMM, TE_OP_DENSE_FP4_FWD,
 TE_OP_DENSE_FP4_BWD) = range(12)
TE_MXFP8, TE_MXFP4, TE_NVFP4 = range(3)

NORM_TYPES = {"layernorm": TE_LAYERNORM, "rmsnorm": TE_RMSNORM}
ACT_TYPES = {"identity": TE_IDENTITY, "relu": TE_RELU, "gelu": TE_GELU, "silu": TE_SILU,
             "swiglu": TE_SWIGLU, "geglu": TE_GEGLU, "reglu": TE_REGLU}
# the pages' activation_type tuples
ACT_TUPLES = {("relu",): "relu", ("gelu",): "gelu", ("silu",): "silu",
              ("silu", "linear"): "swiglu", ("gelu", "linear"): "geglu",
              ("relu", "linear"): "reglu"}
BLOCK_FORMATS = {"mxfp8": TE_MXFP8, "mxfp4": TE_MXFP4, "nvfp4": TE_NVFP4}

_DTYPE = {torch.float32: TE_F32, torch.bfloat16: TE_BF16, torch.uint8: TE_E4M3,
          torch.float8_e4m3fn: TE_E4M3}

EXPORTED = ["te_status_string", "te_version", "te_get_device_status", "te_workspace_size",
            "te_norm_fwd", "te_act_lu", "te_dact_dbias_quantize", "te_quantize", "te_gemm",
            "te_layernorm_dense_fwd", "te_layernorm_mlp_fwd", "te_norm_bwd",
            "te_profile_begin", "te_profile_end", "te_layernorm_mlp_bwd",
            "te_layernorm_dense_bwd",
            "te_dact_dbias_quantize_noalloc",
            "te_dact_dbias_noalloc_capacity", "te_selftest_wait_timeout",
            "te_layernorm_mlp_fwd_host", "te_update_scales", "te_stream_probe",
            "te_block_scale_bytes", "te_block_quantize", "te_block_dequantize", "te_block_gemm",
            "te_dense_fp4_fwd", "te_dense_fp4_bwd", "te_dact_dbias_ckpt"]
KERNEL_KINDS = ["norm_fwd", "quantize", "act_lu", "dact_dbias", "gemm", "gemm_act", "norm_bwd",
                "transpose"]


class TEError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {msg}")
        self.status = status


class _Quantizer(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_void_p), ("scale_inv", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("mode", ctypes.c_int32)]


class _QuantizerSet(ctypes.Structure):
    _fields_ = [("x", _Quantizer), ("kernel1", _Quantizer), ("act", _Quantizer),
                ("kernel2", _Quantizer), ("grad", _Quantizer)]


_lib = None
_lock = threading.Lock()

_vp, _i64, _f, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int32, ctypes.c_size_t
_QP = ctypes.POINTER(_Quantizer)
_QSP = ctypes.POINTER(_QuantizerSet)

_SIGS = {
    "te_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "te_version": (ctypes.c_int, []),
    "te_get_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32)]),
    "te_workspace_size": (_sz, [ctypes.c_int, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                ctypes.c_int, ctypes.c_int]),
    "te_norm_fwd": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _vp, _vp, ctypes.c_int,
                                   ctypes.c_int, _f, _QP, _vp, ctypes.c_int, _vp, _vp, _vp]),
    "te_act_lu": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, ctypes.c_int, _QP, _vp,
                                 ctypes.c_int, _vp]),
    "te_dact_dbias_quantize": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, ctypes.c_int,
                                              _QP, _vp, ctypes.c_int, _vp, _vp, _sz, _vp]),
    "te_quantize": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _QP, _vp, _vp]),
    "te_gemm": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_int, ctypes.c_int, _i64, _i64,
                               _i64, _vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _sz,
                               _vp]),
    "te_layernorm_dense_fwd": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                                              ctypes.c_int, ctypes.c_int, _f, _QSP, _i64, _i64,
                                              _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _sz,
                                              _vp]),
    "te_layernorm_mlp_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp,
                                            ctypes.c_int, ctypes.c_int, _f, ctypes.c_int, _QSP,
                                            _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp,
                                            _vp, _vp, _vp, _sz, _vp]),
    "te_norm_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, ctypes.c_int, _i64, _i64,
                                   ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_profile_begin": (ctypes.c_int, [ctypes.c_int32]),
    "te_layernorm_mlp_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                                            _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _QSP,
                                            _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp,
                                            _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_selftest_wait_timeout": (ctypes.c_int, [_i64, _vp]),
    "te_layernorm_mlp_fwd_host": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int,
                                                 ctypes.c_int, ctypes.c_float, ctypes.c_int, _i64,
                                                 _i64, _i64, ctypes.c_int, _vp, ctypes.c_int, _vp,
                                                 _sz, _vp]),
    "te_layernorm_dense_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                                              ctypes.c_int, ctypes.c_int, _QSP, _i64, _i64, _i64,
                                              ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                              _vp]),
    "te_dact_dbias_quantize_noalloc": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64,
                                                      ctypes.c_int, _QP, _vp, ctypes.c_int, _vp,
                                                      _vp]),
    "te_dact_dbias_noalloc_capacity": (_sz, []),
    "te_profile_end": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int32)]),
    "te_update_scales": (ctypes.c_int, [_QP, ctypes.c_int, _vp]),
    "te_stream_probe": (ctypes.c_int, [_vp, _vp, _sz, ctypes.c_int, _sz, _vp]),
    "te_block_scale_bytes": (_sz, [ctypes.c_int, _i64, _i64]),
    "te_block_quantize": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, ctypes.c_int, _QP, _vp, _vp,
                                         _vp, _vp, _vp]),
    "te_block_dequantize": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _i64, _i64, _vp,
                                           ctypes.c_int, _vp]),
    "te_block_gemm": (ctypes.c_int, [_vp, _vp, _vp, _vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp,
                                     _vp, ctypes.c_int, _vp, ctypes.c_int, _vp]),
    "te_dense_fp4_fwd": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _QP, _vp, _vp,
                                        _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_dense_fp4_bwd": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _vp, _vp, ctypes.c_int, _QP,
                                        _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_dact_dbias_ckpt": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i64, _i64, ctypes.c_int,
                                          _QP, _vp, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
}


def lib_path() -> str:
    return _build.LIB_PATH


def lib(build_if_stale: bool = True) -> ctypes.CDLL:
    """The loaded library; compiles it first when it is missing or older than its sources."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_stale and not _build.up_to_date():
                _build.build()
            if not os.path.exists(_build.LIB_PATH):
                raise ImportError(f"{_build.LIB_PATH} is missing: build it with "
                                  "fp8_transformer_gb300.build.build()")
            h = ctypes.CDLL(_build.LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(h, name)
                fn.restype = res
                fn.argtypes = args
            _lib = h
    return _lib


def _check(fn: str, status: int):
    if status != TE_OK:
        msg = lib().te_status_string(status).decode()
        raise TEError(fn, status, msg)


def _host_ptr(t):
    """Host tensor for the host-buffer entry points (pinned memory lets the copies overlap)."""
    if t.is_cuda:
        raise ValueError("this argument is a host buffer")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the CUDA library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _dt(t) -> int:
    return _DTYPE[t.dtype]


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


class Quantizer:
    """Device scalars of one FP8 quantizer (scale, scale_inv, amax) and its scaling mode."""

    def __init__(self, scale=1.0, mode="delayed", device="cuda"):
        self.scale = torch.tensor([float(scale)], dtype=torch.float32, device=device)
        self.scale_inv = torch.tensor([1.0 / float(scale)], dtype=torch.float32, device=device)
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)
        self.mode = TE_SCALING_CURRENT if mode == "current" else TE_SCALING_DELAYED

    @classmethod
    def from_tensors(cls, scale, scale_inv, amax, mode="delayed"):
        """A quantizer over caller-owned one-element fp32 tensors (e.g. views into a bank).
        amax=None with delayed scaling: the call's amax is not kept."""
        q = cls.__new__(cls)
        q.scale, q.scale_inv, q.amax = scale, scale_inv, amax
        q.mode = TE_SCALING_CURRENT if mode == "current" else TE_SCALING_DELAYED
        return q

    def c(self) -> _Quantizer:
        return _Quantizer(self.scale.data_ptr(), self.scale_inv.data_ptr(),
                          None if self.amax is None else self.amax.data_ptr(), self.mode)


class QuantizerSet:
    """The pages' QuantizerSet: quantizers for x, kernel1, act, kernel2 and grad."""

    def __init__(self, x=None, kernel1=None, act=None, kernel2=None, grad=None):
        self.x, self.kernel1, self.act, self.kernel2, self.grad = x, kernel1, act, kernel2, grad

    def c(self) -> _QuantizerSet:
        z = _Quantizer(None, None, None, 0)
        return _QuantizerSet(*(q.c() if q is not None else z
                               for q in (self.x, self.kernel1, self.act, self.kernel2, self.grad)))


def _qp(q):
    return ctypes.byref(q.c()) if q is not None else None


def status_string(status: int) -> str:
    return lib().te_status_string(status).decode()


def version() -> int:
    return lib().te_version()


def get_device_status() -> int:
    v = ctypes.c_int32(0)
    _check("te_get_device_status", lib().te_get_device_status(ctypes.byref(v)))
    return v.value


def selftest_wait_timeout(limit_us: int = 20000, stream=None):
    """Launch the library's bounded-wait self-test: a wait that nothing completes gives up after
    limit_us and records TE_ERR_TIMEOUT, which get_device_status() then returns."""
    _check("te_selftest_wait_timeout", lib().te_selftest_wait_timeout(int(limit_us), _stream(stream)))


def workspace_size(op, M, H, F_or_N, dtype=TE_BF16, quantized=False, kernel_dtype=None,
                   act=TE_IDENTITY) -> int:
    kd = dtype if kernel_dtype is None else kernel_dtype
    return int(lib().te_workspace_size(op, M, H, F_or_N, dtype, int(bool(quantized)), kd, act))


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _act_id(act) -> int:
    if isinstance(act, tuple):
        act = ACT_TUPLES[act]
    return ACT_TYPES[act] if isinstance(act, str) else int(act)


def _norm_id(norm) -> int:
    return NORM_TYPES[norm] if isinstance(norm, str) else int(norm)


# -------------------------------------------------------------------------- entry points ---


def te_norm_fwd(x, gamma, beta, norm_type, zero_centered_gamma, epsilon, out, q=None, mu=None,
                rsigma=None, stream=None):
    M, H = x.shape
    st = lib().te_norm_fwd(_ptr(x), _dt(x), M, H, _ptr(gamma), _ptr(beta), _norm_id(norm_type),
                           int(bool(zero_centered_gamma)), float(epsilon), _qp(q), _ptr(out),
                           _dt(out), _ptr(mu), _ptr(rsigma), _stream(stream))
    _check("te_norm_fwd", st)
    return out


def te_act_lu(x, act, out, q=None, stream=None):
    M, N_in = x.shape
    st = lib().te_act_lu(_ptr(x), _dt(x), M, N_in, _act_id(act), _qp(q), _ptr(out), _dt(out),
                         _stream(stream))
    _check("te_act_lu", st)
    return out


def te_dact_dbias_quantize(dy, x_preact, act, dx, dbias=None, q=None, workspace=None,
                           stream=None):
    M, N_in = dx.shape
    a = _act_id(act)
    if dbias is not None and workspace is None:
        workspace = _ws(workspace_size(TE_OP_DACT_DBIAS, M, 0, N_in), dx.device)
    st = lib().te_dact_dbias_quantize(_ptr(dy), _ptr(x_preact), _dt(dy), M, N_in, a, _qp(q),
                                      _ptr(dx), _dt(dx), _ptr(dbias), _ptr(workspace),
                                      0 if workspace is None else workspace.numel(),
                                      _stream(stream))
    _check("te_dact_dbias_quantize", st)
    return dx


def te_quantize(x, q, out, stream=None):
    M, N = x.shape if x.dim() == 2 else (1, x.numel())
    st = lib().te_quantize(_ptr(x), _dt(x), M, N, _qp(q), _ptr(out), _stream(stream))
    _check("te_quantize", st)
    return out


def te_gemm(A, B, out, a_trans=False, b_trans=False, a_scale_inv=None, b_scale_inv=None,
            bias=None, workspace=None, split_k=True, stream=None):
    """split_k=False passes no workspace: no tile is split along K."""
    M = A.shape[1] if a_trans else A.shape[0]
    K = A.shape[0] if a_trans else A.shape[1]
    N = B.shape[0] if b_trans else B.shape[1]
    if workspace is None and split_k:
        n = workspace_size(TE_OP_GEMM, M, K, N, _dt(A))
        workspace = _ws(n, A.device) if n > 0 else None
    st = lib().te_gemm(_ptr(A), int(bool(a_trans)), _ptr(B), int(bool(b_trans)), _dt(A), M, N, K,
                       _ptr(a_scale_inv), _ptr(b_scale_inv), _ptr(bias),
                       _dt(bias) if bias is not None else TE_F32, _ptr(out), _dt(out),
                       _ptr(workspace), 0 if workspace is None else workspace.numel(),
                       _stream(stream))
    _check("te_gemm", st)
    return out


def te_layernorm_dense_fwd(x, kernel, gamma, beta, bias, out, norm_type="layernorm",
                           zero_centered_gamma=False, epsilon=1e-6, quantizer_set=None,
                           saved_ln_out=None, mu=None, rsigma=None, workspace=None, stream=None):
    M, H = x.shape
    N = kernel.shape[1]
    dt = _dt(x)
    kd = _dt(kernel)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_DENSE_FWD, M, H, N, dt,
                                       quantizer_set is not None, kd), x.device)
    qs = quantizer_set.c() if quantizer_set is not None else None
    st = lib().te_layernorm_dense_fwd(_ptr(x), _ptr(kernel), kd, _ptr(gamma), _ptr(beta),
                                      _ptr(bias), _norm_id(norm_type), int(bool(zero_centered_gamma)),
                                      float(epsilon), ctypes.byref(qs) if qs is not None else None,
                                      M, H, N, dt, _ptr(out), _ptr(saved_ln_out), _ptr(mu),
                                      _ptr(rsigma), _ptr(workspace), workspace.numel(),
                                      _stream(stream))
    _check("te_layernorm_dense_fwd", st)
    return out


def te_layernorm_mlp_fwd(x, gamma, beta, kernel1, kernel2, bias1, bias2, out,
                         norm_type="layernorm", zero_centered_gamma=False, epsilon=1e-6,
                         activation_type=("relu",), quantizer_set=None, saved_h=None,
                         saved_ln_out=None, mu=None, rsigma=None, workspace=None, stream=None,
                         saved_act=None):
    M, H = x.shape
    F = kernel2.shape[0]
    act = _act_id(activation_type)
    dt = _dt(x)
    kd = _dt(kernel1)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_MLP_FWD, M, H, F, dt,
                                       quantizer_set is not None, kd, act), x.device)
    qs = quantizer_set.c() if quantizer_set is not None else None
    st = lib().te_layernorm_mlp_fwd(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(kernel1),
                                    _ptr(kernel2), kd, _ptr(bias1), _ptr(bias2),
                                    _norm_id(norm_type), int(bool(zero_centered_gamma)),
                                    float(epsilon), act,
                                    ctypes.byref(qs) if qs is not None else None, M, H, F, dt,
                                    _ptr(out), _ptr(saved_h), _ptr(saved_act),
                                    _ptr(saved_ln_out), _ptr(mu), _ptr(rsigma), _ptr(workspace),
                                    workspace.numel(), _stream(stream))
    _check("te_layernorm_mlp_fwd", st)
    return out


def te_layernorm_mlp_fwd_host(x_host, gamma, beta, kernel1, kernel2, bias1, bias2, out_host,
                              norm_type="layernorm", zero_centered_gamma=False, epsilon=1e-6,
                              activation_type=("relu",), chunks=4, workspace=None, stream=None):
    """te_layernorm_mlp_fwd with x and out in (pinned) host memory, copies overlapped with the
    compute of other row slices; the weights are device tensors."""
    M, H = x_host.shape
    F = kernel2.shape[0]
    act = _act_id(activation_type)
    dt = _dt(x_host)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_MLP_FWD_HOST, M, H, F, dt, False, dt, act),
                        kernel1.device)
    st = lib().te_layernorm_mlp_fwd_host(_host_ptr(x_host), _ptr(gamma), _ptr(beta), _ptr(kernel1),
                                         _ptr(kernel2), _ptr(bias1), _ptr(bias2),
                                         _norm_id(norm_type), int(bool(zero_centered_gamma)),
                                         float(epsilon), act, M, H, F, dt, _host_ptr(out_host),
                                         int(chunks), _ptr(workspace), workspace.numel(),
                                         _stream(stream))
    _check("te_layernorm_mlp_fwd_host", st)
    return out_host


def te_layernorm_mlp_bwd(dy, x, gamma, kernel1, kernel2, saved_h, saved_ln_out, mu, rsigma,
                         dx, dgamma, dkernel1, dkernel2, dbeta=None, dbias1=None, dbias2=None,
                         norm_type="layernorm", zero_centered_gamma=False,
                         activation_type=("relu",), quantizer_set=None, workspace=None,
                         stream=None, saved_dh=None):
    M, H = x.shape
    F = kernel2.shape[0]
    act = _act_id(activation_type)
    dt = _dt(x)
    kd = _dt(kernel1)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_MLP_BWD, M, H, F, dt,
                                       quantizer_set is not None, kd, act), x.device)
    qs = quantizer_set.c() if quantizer_set is not None else None
    st = lib().te_layernorm_mlp_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(kernel1), _ptr(kernel2),
                                    kd, _ptr(saved_h), _ptr(saved_ln_out), _ptr(mu), _ptr(rsigma),
                                    _norm_id(norm_type), int(bool(zero_centered_gamma)), act,
                                    ctypes.byref(qs) if qs is not None else None, M, H, F, dt,
                                    _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(dkernel1),
                                    _ptr(dkernel2), _ptr(dbias1), _ptr(dbias2), _ptr(saved_dh),
                                    _ptr(workspace), workspace.numel(), _stream(stream))
    _check("te_layernorm_mlp_bwd", st)
    return dx


def te_layernorm_dense_bwd(dy, x, gamma, kernel, saved_ln_out, mu, rsigma, dx, dgamma, dkernel,
                           dbeta=None, dbias=None, norm_type="layernorm", zero_centered_gamma=False,
                           quantizer_set=None, workspace=None, stream=None):
    M, H = x.shape
    N = kernel.shape[1]
    dt = _dt(x)
    kd = _dt(kernel)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_DENSE_BWD, M, H, N, dt,
                                       quantizer_set is not None, kd), x.device)
    qs = quantizer_set.c() if quantizer_set is not None else None
    st = lib().te_layernorm_dense_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(kernel), kd,
                                      _ptr(saved_ln_out), _ptr(mu), _ptr(rsigma),
                                      _norm_id(norm_type), int(bool(zero_centered_gamma)),
                                      ctypes.byref(qs) if qs is not None else None, M, H, N, dt,
                                      _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(dkernel),
                                      _ptr(dbias), _ptr(workspace), workspace.numel(),
                                      _stream(stream))
    _check("te_layernorm_dense_bwd", st)
    return dx


def te_norm_bwd(dz, x, mu, rsigma, gamma, norm_type, zero_centered_gamma, dx, dgamma,
                dbeta=None, workspace=None, stream=None):
    M, H = x.shape
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_NORM_BWD, M, H, 0), x.device)
    st = lib().te_norm_bwd(_ptr(dz), _ptr(x), _ptr(mu), _ptr(rsigma), _ptr(gamma), _dt(x), M, H,
                           _norm_id(norm_type), int(bool(zero_centered_gamma)), _ptr(dx),
                           _ptr(dgamma), _ptr(dbeta), _ptr(workspace), workspace.numel(),
                           _stream(stream))
    _check("te_norm_bwd", st)
    return dx


def profile_begin(max_records: int = 4096):
    """Start timing every library kernel launch with CUDA events on its launching stream."""
    _check("te_profile_begin", lib().te_profile_begin(int(max_records)))


def stream_probe(src, dst=None, write_bytes=0, ratio=1, read_only_bytes=0, stream=None):
    """One launch of the library's streaming reference kernel (te_stream_probe)."""
    _check("te_stream_probe", lib().te_stream_probe(_ptr(src), _ptr(dst), int(write_bytes),
                                                     int(ratio), int(read_only_bytes),
                                                     _stream(stream)))


def profile_end() -> dict:
    """Stop timing; returns {kind: (total_ms, launches)} for the kernels launched since begin."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int32 * n)()
    _check("te_profile_end", lib().te_profile_end(ms, cnt))
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}


def te_update_scales(quantizers, stream=None):
    """scale = 448 / amax and scale_inv = 1 / scale on the device for every given quantizer
    (the delayed-scaling update between calls, e.g. after an amax all-reduce)."""
    qs = [q for q in quantizers if q is not None]
    arr = (_Quantizer * max(len(qs), 1))(*(q.c() for q in qs))
    _check("te_update_scales", lib().te_update_scales(arr, len(qs), _stream(stream)))


def te_dact_dbias_quantize_noalloc(dy, x_preact, act, dx, dbias=None, q=None, stream=None):
    """te_dact_dbias_quantize without a workspace: the bias reduction uses the library's fixed
    device scratch (see include/te_gb300.h for its capacity and sharing rules)."""
    M, N_in = dx.shape
    st = lib().te_dact_dbias_quantize_noalloc(_ptr(dy), _ptr(x_preact), _dt(dy), M, N_in,
                                              _act_id(act), _qp(q), _ptr(dx), _dt(dx),
                                              _ptr(dbias), _stream(stream))
    _check("te_dact_dbias_quantize_noalloc", st)
    return dx


def dact_dbias_noalloc_capacity() -> int:
    """Floats of fixed device scratch behind te_dact_dbias_quantize_noalloc."""
    return int(lib().te_dact_dbias_noalloc_capacity())


# ------------------------------------------------------------------- block-scaled tensors ---


def _format(fmt) -> int:
    return BLOCK_FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _on_device(*tensors):
    """The tensors (None left out) lie on the current device, where the kernels are launched."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != dev:
            raise ValueError(f"tensors must live on the current device (cuda:{dev})")


def _expect(name, t, shape, *dtypes):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")


_ACT_DTYPES = (torch.float32, torch.bfloat16)
_BYTES = (torch.uint8, torch.float8_e4m3fn)


def block_scale_bytes(fmt, rows, cols) -> int:
    """Bytes of the scales of a [rows, cols] tensor packed along its columns."""
    return int(lib().te_block_scale_bytes(_format(fmt), int(rows), int(cols)))


def block_empty(fmt, rows, cols, device="cuda"):
    """(codes, scales): uninitialized buffers for a [rows, cols] tensor packed along its columns."""
    f = _format(fmt)
    codes = torch.empty(rows, cols if f == TE_MXFP8 else cols // 2, dtype=torch.uint8, device=device)
    return codes, torch.empty(block_scale_bytes(f, rows, cols), dtype=torch.uint8, device=device)


def _expect_packed(name, f, codes, scales, rows, cols):
    _expect(name, codes, (rows, cols if f == TE_MXFP8 else cols // 2),
            *(_BYTES if f == TE_MXFP8 else _BYTES[:1]))
    if scales is None or scales.dtype not in _BYTES or \
            scales.numel() < lib().te_block_scale_bytes(f, rows, cols):
        raise ValueError(f"{name}: its scales must be uint8 of at least block_scale_bytes(fmt, {rows}, {cols})")


def _expect_scalar(name, t):
    if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
        raise ValueError(f"{name}: a one-element float32 tensor")


def _expect_quantizer(f, q):
    if (f == TE_NVFP4) != (q is not None):
        raise ValueError("q: the quantizer of nvfp4's tensor scale (None for the other formats)")
    if q is not None:
        for name in ("scale", "scale_inv", "amax"):
            _expect_scalar(f"q.{name}", getattr(q, name))
        _on_device(q.scale, q.scale_inv, q.amax)


def _workspace_for(op, M, H, N, device, workspace, stream):
    if workspace is None:
        workspace = _ws(workspace_size(op, M, H, N), device)
        if stream is not None:  # freed on return: kept from reuse until that stream has passed it
            workspace.record_stream(stream)
    return workspace


def te_block_quantize(x, fmt, codes=None, scales=None, codes_t=None, scales_t=None, q=None, stream=None):
    """Pack x [M, N] along N into codes / scales, and (or) x^T [N, M rounded up to 32] along M into
    codes_t / scales_t, in one pass.  fmt: "mxfp8", "mxfp4" or "nvfp4" (with q, its tensor scale)."""
    f = _format(fmt)
    M, N = x.shape
    _expect("x", x, (M, N), *_ACT_DTYPES)
    if codes is not None:
        _expect_packed("codes", f, codes, scales, M, N)
    if codes_t is not None:
        _expect_packed("codes_t", f, codes_t, scales_t, N, (M + 31) // 32 * 32)
    _expect_quantizer(f, q)
    _on_device(x, codes, scales, codes_t, scales_t)
    st = lib().te_block_quantize(_ptr(x), _dt(x), M, N, f, _qp(q), _ptr(codes), _ptr(scales),
                                 _ptr(codes_t), _ptr(scales_t), _stream(stream))
    _check("te_block_quantize", st)


def te_block_dequantize(codes, scales, fmt, out, scale_inv=None, stream=None):
    """out [M, N] (float32 / bfloat16): the values that packed codes stand for."""
    f = _format(fmt)
    M, N = out.shape
    _expect("out", out, (M, N), *_ACT_DTYPES)
    _expect_packed("codes", f, codes, scales, M, N)
    _expect_scalar("scale_inv", scale_inv)
    _on_device(codes, scales, out, scale_inv)
    st = lib().te_block_dequantize(_ptr(codes), _ptr(scales), f, _ptr(scale_inv), M, N, _ptr(out),
                                   _dt(out), _stream(stream))
    _check("te_block_dequantize", st)
    return out


def te_block_gemm(a, a_scales, b, b_scales, out, fmt, a_scale_inv=None, b_scale_inv=None, bias=None,
                  stream=None):
    """out [M, N] = alpha * A B^T + bias of packed 4-bit operands a [M, K / 2] and b [N, K / 2]."""
    f = _format(fmt)
    M, N = out.shape
    K = 2 * a.shape[1]
    _expect("out", out, (M, N), *_ACT_DTYPES)
    _expect_packed("a", f, a, a_scales, M, K if f != TE_MXFP8 else K // 2)
    _expect_packed("b", f, b, b_scales, N, K if f != TE_MXFP8 else K // 2)
    if bias is not None:
        _expect("bias", bias, (N,), *_ACT_DTYPES)
    _expect_scalar("a_scale_inv", a_scale_inv)
    _expect_scalar("b_scale_inv", b_scale_inv)
    _on_device(a, a_scales, b, b_scales, out, a_scale_inv, b_scale_inv, bias)
    st = lib().te_block_gemm(_ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales), f, M, N, K,
                             _ptr(a_scale_inv), _ptr(b_scale_inv), _ptr(bias),
                             _dt(bias) if bias is not None else TE_F32, _ptr(out), _dt(out),
                             _stream(stream))
    _check("te_block_gemm", st)
    return out


def te_dense_fp4_fwd(x, kernel, kernel_scales, out, fmt, bias=None, q=None, kernel_scale_inv=None,
                     saved_xt=None, saved_xt_scales=None, workspace=None, stream=None):
    """out [M, N] = x [M, K] @ kernel + bias with x packed on the way; kernel: [N, K / 2], the
    transposed codes (codes_t) of a kernel stored [K, N]."""
    f = _format(fmt)
    M, K = x.shape
    N = out.shape[1]
    _expect("x", x, (M, K), *_ACT_DTYPES)
    _expect("out", out, (M, N), x.dtype)
    _expect_packed("kernel", f, kernel, kernel_scales, N, K)
    if bias is not None:
        _expect("bias", bias, (N,), x.dtype)
    if saved_xt is not None:
        _expect_packed("saved_xt", f, saved_xt, saved_xt_scales, K, (M + 31) // 32 * 32)
    _expect_quantizer(f, q)
    _expect_scalar("kernel_scale_inv", kernel_scale_inv)
    _on_device(x, kernel, kernel_scales, out, bias, kernel_scale_inv, saved_xt, saved_xt_scales, workspace)
    workspace = _workspace_for(TE_OP_DENSE_FP4_FWD, M, K, N, x.device, workspace, stream)
    st = lib().te_dense_fp4_fwd(_ptr(x), _dt(x), _ptr(kernel), _ptr(kernel_scales), f, _qp(q),
                                _ptr(kernel_scale_inv), _ptr(bias), M, K, N, _ptr(out),
                                _ptr(saved_xt), _ptr(saved_xt_scales), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check("te_dense_fp4_fwd", st)
    return out


def te_dense_fp4_bwd(dy, kernel, kernel_scales, saved_xt, saved_xt_scales, dx, dkernel, fmt, dbias=None,
                     q=None, kernel_scale_inv=None, x_scale_inv=None, workspace=None, stream=None):
    """dx = dy @ kernel^T, dkernel [K, N] = x^T @ dy and dbias from 4-bit operands; kernel: [K, N / 2],
    the codes of a kernel stored [K, N]; saved_xt from te_dense_fp4_fwd."""
    f = _format(fmt)
    M, N = dy.shape
    K = dx.shape[1]
    _expect("dy", dy, (M, N), *_ACT_DTYPES)
    _expect("dx", dx, (M, K), dy.dtype)
    _expect("dkernel", dkernel, (K, N), dy.dtype)
    _expect_packed("kernel", f, kernel, kernel_scales, K, N)
    _expect_packed("saved_xt", f, saved_xt, saved_xt_scales, K, (M + 31) // 32 * 32)
    if dbias is not None:
        _expect("dbias", dbias, (N,), torch.float32)
    _expect_quantizer(f, q)
    _expect_scalar("kernel_scale_inv", kernel_scale_inv)
    _expect_scalar("x_scale_inv", x_scale_inv)
    _on_device(dy, kernel, kernel_scales, saved_xt, saved_xt_scales, dx, dkernel, dbias, kernel_scale_inv,
               x_scale_inv, workspace)
    workspace = _workspace_for(TE_OP_DENSE_FP4_BWD, M, K, N, dy.device, workspace, stream)
    st = lib().te_dense_fp4_bwd(_ptr(dy), _dt(dy), _ptr(kernel), _ptr(kernel_scales), _ptr(saved_xt),
                                _ptr(saved_xt_scales), f, _qp(q), _ptr(kernel_scale_inv),
                                _ptr(x_scale_inv), M, K, N, _ptr(dx), _ptr(dkernel), _ptr(dbias),
                                _ptr(workspace), workspace.numel(), _stream(stream))
    _check("te_dense_fp4_bwd", st)
    return dx


def te_dact_dbias_ckpt(dy, codes, scales, act, dx, dbias=None, act_out=None, q=None, workspace=None,
                       stream=None):
    """te_dact_dbias_quantize from an 8-bit checkpoint (codes, scales: mxfp8) of the activation's
    input; act_out, when given, receives the recomputed activation output."""
    a = _act_id(act)
    M, N_in = dx.shape
    n_out = N_in // 2 if a in (TE_SWIGLU, TE_GEGLU, TE_REGLU) else N_in
    _expect("dy", dy, (M, n_out), *_ACT_DTYPES)
    _expect("dx", dx, (M, N_in), *_ACT_DTYPES, *_BYTES)
    _expect_packed("codes", TE_MXFP8, codes, scales, M, N_in)
    if act_out is not None:
        _expect("act_out", act_out, (M, n_out), dy.dtype)
    if dbias is not None:
        _expect("dbias", dbias, (N_in,), torch.float32)
        workspace = _workspace_for(TE_OP_DACT_DBIAS, M, 0, N_in, dy.device, workspace, stream)
    _on_device(dy, codes, scales, dx, dbias, act_out, workspace)
    st = lib().te_dact_dbias_ckpt(_ptr(dy), _ptr(codes), _ptr(scales), _dt(dy), M, N_in, a, _qp(q),
                                  _ptr(dx), _dt(dx), _ptr(act_out), _ptr(dbias), _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _stream(stream))
    _check("te_dact_dbias_ckpt", st)
    return dx

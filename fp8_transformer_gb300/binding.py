"""ctypes binding of libte_gb300.so (the C ABI declared in include/te_gb300.h).

Argument marshalling only: each function takes torch tensors, checks their dtype/shape against
the C signature, and passes raw device pointers and sizes.  Every step of the computation runs
in the library's CUDA kernels; there is no fallback.  A missing or unbuildable library raises.
"""

from __future__ import annotations

import ctypes
import functools
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
            "te_selftest_cluster_abort",
            "te_layernorm_mlp_fwd_host", "te_update_scales", "te_stream_probe",
            "te_block_scale_bytes", "te_block_quantize", "te_block_dequantize", "te_block_gemm",
            "te_dense_fp4_fwd", "te_dense_fp4_bwd", "te_dact_dbias_ckpt",
            "te_layernorm_mlp_fwd_ckpt", "te_layernorm_mlp_bwd_ckpt",
            "te_residual_norm_fwd", "te_residual_norm_bwd", "te_residual_norm_bwd_workspace",
            "te_dense_residual_fwd", "te_dense_residual_fwd_workspace", "te_dense_residual_bwd",
            "te_dense_residual_bwd_workspace", "te_grad_norm", "te_clip_grad_norm",
            "te_grad_norm_workspace"]
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


class _Grad(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


_lib = None
_read_grads = None  # of the library that reads tensors
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
    "te_selftest_cluster_abort": (ctypes.c_int, [_i64, ctypes.c_int, _vp, _vp]),
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
_int, _GP = ctypes.c_int, ctypes.POINTER(_Grad)
_SIGS.update({
    "te_residual_norm_fwd": (_int, [_vp, _int, _vp, _int, _i64, _i64] + [_vp] * 5 + [_i64, _f, _int, _int, _f, _QP,
                                    _vp, _vp, _int] + [_vp] * 5),
    "te_residual_norm_bwd_workspace": (_sz, [_i64] * 3),
    "te_residual_norm_bwd": (_int, [_vp] * 4 + [_int, _int, _i64, _i64] + [_vp] * 8 + [_i64, _f, _int, _int]
                             + [_vp] * 8 + [_sz, _vp]),
    "te_dense_residual_fwd_workspace": (_sz, [_i64] * 3 + [_int]),
    "te_dense_residual_fwd": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _int, _vp, _i64, _vp, _int, _f, _i64, _i64, _i64,
                                     _vp, _vp, _vp, _sz, _vp]),
    "te_dense_residual_bwd_workspace": (_sz, [_i64] * 4 + [_int]),
    "te_dense_residual_bwd": (_int, [_vp, _int, _vp, _vp, _int, _vp, _int, _vp, _i64, _f, _QP, _vp, _vp, _i64, _i64,
                                     _i64] + [_vp] * 6 + [_sz, _vp]),
    "te_grad_norm_workspace": (_sz, [_i64]),
    "te_grad_norm": (_int, [_GP, _i64, _vp, _vp, _sz, _vp]),
    "te_clip_grad_norm": (_int, [_GP, _i64, ctypes.c_double, ctypes.c_double, _vp, _vp, _sz, _vp]),
})
# the checkpoint forms have two pointers (codes, scales) in the place of saved_h
for _name, _at in (("te_layernorm_mlp_fwd", 17), ("te_layernorm_mlp_bwd", 6)):
    _res, _args = _SIGS[_name]
    _SIGS[_name + "_ckpt"] = (_res, _args[:_at] + [_vp] + _args[_at:])


def lib_path() -> str:
    return _build.LIB_PATH


def lib(build_if_stale: bool = True) -> ctypes.CDLL:
    """The loaded library; compiles it first when it is missing or older than its sources."""
    global _lib, _read_grads
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if build_if_stale and not _build.up_to_date():
                _build.build()
            for path in (_build.LIB_PATH, _build.TENSOR_LIB_PATH):
                if not os.path.exists(path):
                    raise ImportError(f"{path} is missing: build it with "
                                      "fp8_transformer_gb300.build.build()")
            _read_grads = ctypes.PyDLL(_build.TENSOR_LIB_PATH).te_read_grads
            _read_grads.restype = _i64
            _read_grads.argtypes = [ctypes.py_object, ctypes.py_object, _i64, _GP, ctypes.POINTER(_i64)]
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


# The raw handle of a device's current stream without building a Stream object for it (2.9 us of a
# call's host time on a Grace core).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if dev is None else dev)
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


def selftest_cluster_abort(out, rank, limit_us: int = 20000, stream=None):
    """The same wait in CTA `rank` (-1: in none) of a cluster; out (8 int32) receives 1 for each of its CTAs that
    would still write results."""
    _check("te_selftest_cluster_abort", lib().te_selftest_cluster_abort(
        int(limit_us), int(rank), _arg("out", out, (8,), (torch.int32,), torch.cuda.current_device()), _stream(stream)))


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


# The checks below run on every call and each call is short, so they are written for few Python
# operations: one pass over a tensor's properties, which also yields its address.

_ACT_DTYPES = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_E4M3_BYTES = (torch.uint8, torch.float8_e4m3fn)
_OUT_DTYPES = _ACT_DTYPES + _E4M3_BYTES
_BF16 = (torch.bfloat16,)
_GEMM_DTYPES = _BF16 + _E4M3_BYTES


def _format(fmt) -> int:
    return BLOCK_FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _arg(name, t, shape, dtypes, dev):
    """Address of a tensor that is on the current device `dev`, dense, and of this shape and type."""
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensors must live on the current device (cuda:{dev})")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _scale_size(f, rows, cols):
    return (rows + 127) // 128 * ((cols // (16 if f == TE_NVFP4 else 32) + 3) // 4) * 512


def _packed(name, codes, scales, f, rows, cols, dev):
    """Addresses of a packed [rows, cols] tensor's codes and scales."""
    if f == TE_MXFP8:
        c = _arg(name, codes, (rows, cols), _E4M3_BYTES, dev)
    else:
        c = _arg(name, codes, (rows, cols // 2), _U8, dev)
    if scales is None or scales.dtype not in _E4M3_BYTES or scales.numel() < _scale_size(f, rows, cols) \
            or scales.get_device() != dev or not scales.is_contiguous():
        raise ValueError(f"{name}: its scales must be dense uint8 on cuda:{dev}, at least "
                         f"block_scale_bytes(fmt, {rows}, {cols}) of them")
    return c, scales.data_ptr()


def _scalar(name, t, dev):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or t.get_device() != dev:
        raise ValueError(f"{name}: a one-element float32 tensor on cuda:{dev}")
    return t.data_ptr()


def _tensor_scale(f, q, dev):
    """The C quantizer of NVFP4's tensor scale (None for the MX formats)."""
    if (f == TE_NVFP4) != (q is not None):
        raise ValueError("q: the quantizer of nvfp4's tensor scale (None for the other formats)")
    if q is None:
        return None
    return ctypes.byref(_quantizer("q", q, dev))


def _quantizer(name, q, dev):
    """The C quantizer, its scalars on the current device (None without one)."""
    if q is None:
        return None
    return _Quantizer(_scalar(name + ".scale", q.scale, dev), _scalar(name + ".scale_inv", q.scale_inv, dev),
                      _scalar(name + ".amax", q.amax, dev), q.mode)


def _quantizer_set(qs, dev):
    """The same of a set, by reference."""
    if qs is None:
        return None
    z = _Quantizer(None, None, None, 0)
    return ctypes.byref(_QuantizerSet(*(_quantizer(k, getattr(qs, k), dev) or z
                                        for k in ("x", "kernel1", "act", "kernel2", "grad"))))


def _sized_arg(name, t, n, dtypes, dev):
    """Address of a tensor of n values in any shape, or None without it."""
    return None if t is None else _arg(name, t.reshape(-1) if t.is_contiguous() else t, (n,), dtypes, dev)


def _given_workspace(workspace, dev):
    """(address, bytes) of a caller's workspace: dense, of any type, on the device `dev` of the other tensors."""
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: dense, on the device of the other tensors")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# (id, device index, device type) of a device's current stream.
_stream_data = torch._C._cuda_getCurrentStream if hasattr(torch._C, "_cuda_getCurrentStream") else None


def _lasting_stream(dev, handle):
    """Whether the current stream of `dev`, of this raw handle, is the default one or of torch's pools:
    these are few and live as long as the process.  A stream made elsewhere has its handle for an id; once
    it is destroyed the handle may come back as another stream's."""
    if handle == 0:
        return True
    sid = torch.cuda.current_stream(dev).stream_id if _stream_data is None else _stream_data(dev)[0]
    return sid != handle


_sized = functools.lru_cache(maxsize=1024)(workspace_size)
_SMALL_WORKSPACE = 1 << 20
_small = threading.local()


def _workspace(op, M, H, N, like, workspace, stream):
    """(tensor, address, bytes) of the given workspace, or of a new one.  Small ones of eager calls
    are kept, one for each host thread and stream of torch's own, whose calls run one after another: an
    allocation costs a short call 5 to 7 us of host time, as much as its launches."""
    return _workspace_of(_sized(op, M, H, N) if workspace is None else 0, like, workspace, stream)


def _workspace_of(n, like, workspace, stream):
    """The same for a size in bytes."""
    if workspace is None:
        n = max(n, 1)
        if n <= _SMALL_WORKSPACE and stream is None and not torch.cuda.is_current_stream_capturing():
            dev = like.get_device()
            key = (dev, _stream(None, dev))
            kept = _small.__dict__.setdefault("kept", {})
            workspace = kept.get(key)
            if workspace is None and _lasting_stream(*key):
                workspace = kept[key] = torch.empty(_SMALL_WORKSPACE, dtype=torch.uint8, device=like.device)
            if workspace is not None:
                return workspace, workspace.data_ptr(), _SMALL_WORKSPACE
        workspace = torch.empty(n, dtype=torch.uint8, device=like.device)
        if stream is not None:  # freed on return: kept from reuse until that stream has passed it
            workspace.record_stream(stream)
    return (workspace, *_given_workspace(workspace, like.get_device()))


def block_scale_bytes(fmt, rows, cols) -> int:
    """Bytes of the scales of a [rows, cols] tensor packed along its columns."""
    return int(lib().te_block_scale_bytes(_format(fmt), int(rows), int(cols)))


def block_empty(fmt, rows, cols, device="cuda"):
    """(codes, scales): uninitialized buffers for a [rows, cols] tensor packed along its columns."""
    f = _format(fmt)
    codes = torch.empty(rows, cols if f == TE_MXFP8 else cols // 2, dtype=torch.uint8, device=device)
    return codes, torch.empty(block_scale_bytes(f, rows, cols), dtype=torch.uint8, device=device)


def te_block_quantize(x, fmt, codes=None, scales=None, codes_t=None, scales_t=None, q=None, stream=None):
    """Pack x [M, N] along N into codes / scales, and (or) x^T [N, M rounded up to 32] along M into
    codes_t / scales_t, in one pass.  fmt: "mxfp8", "mxfp4" or "nvfp4" (with q, its tensor scale)."""
    f, dev = _format(fmt), torch.cuda.current_device()
    M, N = x.shape
    px = _arg("x", x, (M, N), _ACT_DTYPES, dev)
    pc = ps = pct = pst = None
    if codes is not None:
        pc, ps = _packed("codes", codes, scales, f, M, N, dev)
    elif scales is not None:
        raise ValueError("scales: given without their codes")
    if codes_t is not None:
        pct, pst = _packed("codes_t", codes_t, scales_t, f, N, (M + 31) // 32 * 32, dev)
    elif scales_t is not None:
        raise ValueError("scales_t: given without their codes")
    st = lib().te_block_quantize(px, _dt(x), M, N, f, _tensor_scale(f, q, dev), pc, ps, pct, pst,
                                 _stream(stream, dev))
    _check("te_block_quantize", st)


def te_block_dequantize(codes, scales, fmt, out, scale_inv=None, stream=None):
    """out [M, N] (float32 / bfloat16): the values that packed codes stand for."""
    f, dev = _format(fmt), torch.cuda.current_device()
    M, N = out.shape
    po = _arg("out", out, (M, N), _ACT_DTYPES, dev)
    pc, ps = _packed("codes", codes, scales, f, M, N, dev)
    st = lib().te_block_dequantize(pc, ps, f, _scalar("scale_inv", scale_inv, dev), M, N, po, _dt(out),
                                   _stream(stream, dev))
    _check("te_block_dequantize", st)
    return out


def te_block_gemm(a, a_scales, b, b_scales, out, fmt, a_scale_inv=None, b_scale_inv=None, bias=None,
                  stream=None):
    """out [M, N] = alpha * A B^T + bias of packed 4-bit operands a [M, K / 2] and b [N, K / 2]."""
    f, dev = _format(fmt), torch.cuda.current_device()
    M, N = out.shape
    K = a.shape[1] * (1 if f == TE_MXFP8 else 2)
    po = _arg("out", out, (M, N), _ACT_DTYPES, dev)
    pa, psa = _packed("a", a, a_scales, f, M, K, dev)
    pb, psb = _packed("b", b, b_scales, f, N, K, dev)
    pz = None if bias is None else _arg("bias", bias, (N,), _ACT_DTYPES, dev)
    st = lib().te_block_gemm(pa, psa, pb, psb, f, M, N, K, _scalar("a_scale_inv", a_scale_inv, dev),
                             _scalar("b_scale_inv", b_scale_inv, dev), pz,
                             TE_F32 if bias is None else _dt(bias), po, _dt(out), _stream(stream, dev))
    _check("te_block_gemm", st)
    return out


def te_dense_fp4_fwd(x, kernel, kernel_scales, out, fmt, bias=None, q=None, kernel_scale_inv=None,
                     saved_xt=None, saved_xt_scales=None, workspace=None, stream=None):
    """out [M, N] = x [M, K] @ kernel + bias with x packed on the way; kernel: [N, K / 2], the
    transposed codes (codes_t) of a kernel stored [K, N]."""
    f, dev = _format(fmt), torch.cuda.current_device()
    M, K = x.shape
    N = out.shape[1]
    dt = (x.dtype,)
    px = _arg("x", x, (M, K), _ACT_DTYPES, dev)
    po = _arg("out", out, (M, N), dt, dev)
    pk, psk = _packed("kernel", kernel, kernel_scales, f, N, K, dev)
    pz = None if bias is None else _arg("bias", bias, (N,), dt, dev)
    pt = pst = None
    if saved_xt is not None:
        pt, pst = _packed("saved_xt", saved_xt, saved_xt_scales, f, K, (M + 31) // 32 * 32, dev)
    elif saved_xt_scales is not None:
        raise ValueError("saved_xt_scales: given without their codes")
    cq = _tensor_scale(f, q, dev)
    pw, nw = None, 0
    if M > 8 or saved_xt is not None or workspace is not None:
        workspace, pw, nw = _workspace(TE_OP_DENSE_FP4_FWD, M, K, N, x, workspace, stream)
    st = lib().te_dense_fp4_fwd(px, _dt(x), pk, psk, f, cq, _scalar("kernel_scale_inv", kernel_scale_inv, dev),
                                pz, M, K, N, po, pt, pst, pw, nw, _stream(stream, dev))
    _check("te_dense_fp4_fwd", st)
    return out


def te_dense_fp4_bwd(dy, kernel, kernel_scales, saved_xt, saved_xt_scales, dx, dkernel, fmt, dbias=None,
                     q=None, kernel_scale_inv=None, x_scale_inv=None, workspace=None, stream=None):
    """dx = dy @ kernel^T, dkernel [K, N] = x^T @ dy and dbias from 4-bit operands; kernel: [K, N / 2],
    the codes of a kernel stored [K, N]; saved_xt from te_dense_fp4_fwd."""
    f, dev = _format(fmt), torch.cuda.current_device()
    M, N = dy.shape
    K = dx.shape[1]
    dt = (dy.dtype,)
    py = _arg("dy", dy, (M, N), _ACT_DTYPES, dev)
    px = _arg("dx", dx, (M, K), dt, dev)
    pw = _arg("dkernel", dkernel, (K, N), dt, dev)
    pk, psk = _packed("kernel", kernel, kernel_scales, f, K, N, dev)
    pt, pst = _packed("saved_xt", saved_xt, saved_xt_scales, f, K, (M + 31) // 32 * 32, dev)
    pz = None if dbias is None else _arg("dbias", dbias, (N,), _F32, dev)
    cq = _tensor_scale(f, q, dev)
    workspace, pws, nws = _workspace(TE_OP_DENSE_FP4_BWD, M, K, N, dy, workspace, stream)
    st = lib().te_dense_fp4_bwd(py, _dt(dy), pk, psk, pt, pst, f, cq,
                                _scalar("kernel_scale_inv", kernel_scale_inv, dev),
                                _scalar("x_scale_inv", x_scale_inv, dev), M, K, N, px, pw, pz, pws, nws,
                                _stream(stream, dev))
    _check("te_dense_fp4_bwd", st)
    return dx


def te_dact_dbias_ckpt(dy, codes, scales, act, dx, dbias=None, act_out=None, q=None, workspace=None,
                       stream=None):
    """te_dact_dbias_quantize from an 8-bit checkpoint (codes, scales: mxfp8) of the activation's
    input; act_out, when given, receives the recomputed activation output."""
    a, dev = _act_id(act), torch.cuda.current_device()
    M, N_in = dx.shape
    n_out = N_in // 2 if a >= TE_SWIGLU else N_in
    py = _arg("dy", dy, (M, n_out), _ACT_DTYPES, dev)
    px = _arg("dx", dx, (M, N_in), _ACT_DTYPES + _E4M3_BYTES, dev)
    pc, ps = _packed("codes", codes, scales, TE_MXFP8, M, N_in, dev)
    pa = None if act_out is None else _arg("act_out", act_out, (M, n_out), (dy.dtype,), dev)
    pb = pws = None
    nws = 0
    if dbias is not None:
        pb = _arg("dbias", dbias, (N_in,), _F32, dev)
        workspace, pws, nws = _workspace(TE_OP_DACT_DBIAS, M, 0, N_in, dy, workspace, stream)
    cq = None if q is None else ctypes.byref(_quantizer("q", q, dev))
    st = lib().te_dact_dbias_ckpt(py, pc, ps, _dt(dy), M, N_in, a, cq, px, _dt(dx), pa, pb, pws, nws,
                                  _stream(stream, dev))
    _check("te_dact_dbias_ckpt", st)
    return dx


def te_layernorm_mlp_fwd_ckpt(x, gamma, beta, kernel1, kernel2, bias1, bias2, out, h_codes, h_scales,
                              norm_type="layernorm", zero_centered_gamma=False, epsilon=1e-6,
                              activation_type=("relu",), quantizer_set=None, saved_ln_out=None, mu=None,
                              rsigma=None, workspace=None, stream=None, saved_act=None):
    """te_layernorm_mlp_fwd that keeps the activation's input as an 8-bit checkpoint (h_codes, h_scales:
    block_empty("mxfp8", M, F')) for te_layernorm_mlp_bwd_ckpt."""
    M, H = x.shape
    F = kernel2.shape[0]
    act, dt, kd, dev = _act_id(activation_type), _dt(x), _dt(kernel1), torch.cuda.current_device()
    F1 = 2 * F if act >= TE_SWIGLU else F
    pc, ps = _packed("h_codes", h_codes, h_scales, TE_MXFP8, M, F1, dev)
    d = (x.dtype,)
    e = _E4M3_BYTES if quantizer_set is not None else d
    k = _E4M3_BYTES if kd == TE_E4M3 else (kernel1.dtype,)
    px = _arg("x", x, (M, H), _ACT_DTYPES, dev)
    pg, pbe = _sized_arg("gamma", gamma, H, d, dev), _sized_arg("beta", beta, H, d, dev)
    p1, p2 = _sized_arg("kernel1", kernel1, H * F1, k, dev), _sized_arg("kernel2", kernel2, F * H, k, dev)
    pb1, pb2 = _sized_arg("bias1", bias1, F1, d, dev), _sized_arg("bias2", bias2, H, d, dev)
    po = _arg("out", out, (M, H), d, dev)
    pa, pl = _sized_arg("saved_act", saved_act, M * F, e, dev), _sized_arg("saved_ln_out", saved_ln_out, M * H, e, dev)
    pm, pr = _sized_arg("mu", mu, M, _F32, dev), _sized_arg("rsigma", rsigma, M, _F32, dev)
    qs = _quantizer_set(quantizer_set, dev)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_MLP_FWD, M, H, F, dt, quantizer_set is not None, kd, act),
                        x.device)
        if stream is not None:
            workspace.record_stream(stream)
    pw, nw = _given_workspace(workspace, dev)
    st = lib().te_layernorm_mlp_fwd_ckpt(px, pg, pbe, p1, p2, kd, pb1, pb2, _norm_id(norm_type),
                                         int(bool(zero_centered_gamma)), float(epsilon), act, qs, M, H, F, dt, po,
                                         pc, ps, pa, pl, pm, pr, pw, nw,
                                         _stream(stream, dev))
    _check("te_layernorm_mlp_fwd_ckpt", st)
    return out


def te_layernorm_mlp_bwd_ckpt(dy, x, gamma, kernel1, kernel2, h_codes, h_scales, saved_ln_out, mu, rsigma, dx,
                              dgamma, dkernel1, dkernel2, dbeta=None, dbias1=None, dbias2=None,
                              norm_type="layernorm", zero_centered_gamma=False, activation_type=("relu",),
                              quantizer_set=None, workspace=None, stream=None, saved_dh=None):
    """te_layernorm_mlp_bwd from the 8-bit checkpoint that te_layernorm_mlp_fwd_ckpt wrote."""
    M, H = x.shape
    F = kernel2.shape[0]
    act, dt, kd, dev = _act_id(activation_type), _dt(x), _dt(kernel1), torch.cuda.current_device()
    F1 = 2 * F if act >= TE_SWIGLU else F
    pc, ps = _packed("h_codes", h_codes, h_scales, TE_MXFP8, M, F1, dev)
    d = (x.dtype,)
    e = _E4M3_BYTES if quantizer_set is not None else d
    k = _E4M3_BYTES if kd == TE_E4M3 else (kernel1.dtype,)
    py, px = _arg("dy", dy, (M, H), d, dev), _arg("x", x, (M, H), _ACT_DTYPES, dev)
    pg = _sized_arg("gamma", gamma, H, d, dev)
    p1, p2 = _sized_arg("kernel1", kernel1, H * F1, k, dev), _sized_arg("kernel2", kernel2, F * H, d, dev)
    pl = _sized_arg("saved_ln_out", saved_ln_out, M * H, e, dev)
    pm, pr = _sized_arg("mu", mu, M, _F32, dev), _sized_arg("rsigma", rsigma, M, _F32, dev)
    pdx = _arg("dx", dx, (M, H), d, dev)
    pdg, pdb = _sized_arg("dgamma", dgamma, H, _F32, dev), _sized_arg("dbeta", dbeta, H, _F32, dev)
    pd1, pd2 = _sized_arg("dkernel1", dkernel1, H * F1, d, dev), _sized_arg("dkernel2", dkernel2, F * H, d, dev)
    pb1, pb2 = _sized_arg("dbias1", dbias1, F1, _F32, dev), _sized_arg("dbias2", dbias2, H, _F32, dev)
    pdh = _sized_arg("saved_dh", saved_dh, M * F1, e, dev)
    qs = _quantizer_set(quantizer_set, dev)
    if workspace is None:
        workspace = _ws(workspace_size(TE_OP_LAYERNORM_MLP_BWD, M, H, F, dt, quantizer_set is not None, kd, act),
                        x.device)
        if stream is not None:
            workspace.record_stream(stream)
    pw, nw = _given_workspace(workspace, dev)
    st = lib().te_layernorm_mlp_bwd_ckpt(py, px, pg, p1, p2, kd, pc, ps, pl, pm, pr, _norm_id(norm_type),
                                         int(bool(zero_centered_gamma)), act, qs, M, H, F, dt, pdx, pdg, pdb, pd1,
                                         pd2, pb1, pb2, pdh, pw, nw,
                                         _stream(stream, dev))
    _check("te_layernorm_mlp_bwd_ckpt", st)
    return dx


# ------------------------------------------------------------- around the residual stream ---


@functools.lru_cache(maxsize=1024)
def _sized_by(name, *dims):
    return int(getattr(lib(), name)(*dims))


def _gate(gate, M, H, dtypes, dev):
    """(address, rows) of a gate [H] or [G, H] whose rows divide M."""
    g = gate.shape[0] if gate.dim() == 2 else 1
    if gate.dim() == 2:
        p = _arg("gate", gate, (g, H), dtypes, dev)
    else:
        p = _arg("gate", gate, (H,), dtypes, dev)
    if g < 1 or M % g:
        raise ValueError(f"gate: its {g} rows do not divide {M}")
    return p, g


def te_residual_norm_fwd(y, residual, gamma, beta, x_out, out, norm_type="layernorm", zero_centered_gamma=False,
                         epsilon=1e-6, post_gamma=None, post_beta=None, gate=None, residual_scale=1.0, q=None,
                         mu=None, rsigma=None, post_mu=None, post_rsigma=None, stream=None):
    """x_out = residual_scale * residual + gate * p, p = norm(y; post_gamma, post_beta) or y without post_gamma,
    and out = norm(x_out; gamma, beta), in one pass.  gate: [H], or [G, H] with a row for M / G neighbouring
    rows.  x_out may be residual."""
    M, H = y.shape
    dev = torch.cuda.current_device()
    d, r = (y.dtype,), (residual.dtype,)
    py, pr = _arg("y", y, (M, H), _ACT_DTYPES, dev), _arg("residual", residual, (M, H), _ACT_DTYPES, dev)
    h, m = (H,), (M,)
    pg = _arg("gamma", gamma, h, d, dev)
    pb = None if beta is None else _arg("beta", beta, h, d, dev)
    ppg = None if post_gamma is None else _arg("post_gamma", post_gamma, h, d, dev)
    ppb = None if post_beta is None else _arg("post_beta", post_beta, h, d, dev)
    pgt, ng = (None, 1) if gate is None else _gate(gate, M, H, d, dev)
    px = _arg("x_out", x_out, (M, H), r, dev)
    po = _arg("out", out, (M, H), _OUT_DTYPES, dev)
    pm = None if mu is None else _arg("mu", mu, m, _F32, dev)
    prs = None if rsigma is None else _arg("rsigma", rsigma, m, _F32, dev)
    ppm = None if post_mu is None else _arg("post_mu", post_mu, m, _F32, dev)
    pprs = None if post_rsigma is None else _arg("post_rsigma", post_rsigma, m, _F32, dev)
    cq = None if q is None else ctypes.byref(_quantizer("q", q, dev))
    st = lib().te_residual_norm_fwd(py, _dt(y), pr, _dt(residual), M, H, pg, pb, ppg, ppb, pgt, ng,
                                    float(residual_scale), _norm_id(norm_type), int(bool(zero_centered_gamma)),
                                    float(epsilon), cq, px, po, _dt(out), pm, prs, ppm, pprs, _stream(stream, dev))
    _check("te_residual_norm_fwd", st)
    return out


def te_residual_norm_bwd(dout, dx_out, x_out, mu, rsigma, gamma, dresidual, dy, dgamma, dbeta=None, y=None,
                         post_mu=None, post_rsigma=None, post_gamma=None, post_beta=None, gate=None,
                         residual_scale=1.0, dpost_gamma=None, dpost_beta=None, dgate=None, norm_type="layernorm",
                         zero_centered_gamma=False, workspace=None, stream=None):
    """Gradients of te_residual_norm_fwd from dout (of out) and dx_out (what reaches x_out otherwise, or None).
    dresidual (may be dx_out) and dy may be None; y is needed with a post norm or a gate."""
    M, H = dout.shape
    dev = torch.cuda.current_device()
    d, r = (dout.dtype,), (x_out.dtype,)
    mh, h, m = (M, H), (H,), (M,)
    pd = _arg("dout", dout, mh, _ACT_DTYPES, dev)
    pxo = None if dx_out is None else _arg("dx_out", dx_out, mh, r, dev)
    px = _arg("x_out", x_out, mh, _ACT_DTYPES, dev)
    py = None if y is None else _arg("y", y, mh, d, dev)
    pm = None if mu is None else _arg("mu", mu, m, _F32, dev)
    prs = None if rsigma is None else _arg("rsigma", rsigma, m, _F32, dev)
    ppm = None if post_mu is None else _arg("post_mu", post_mu, m, _F32, dev)
    pprs = None if post_rsigma is None else _arg("post_rsigma", post_rsigma, m, _F32, dev)
    pg = _arg("gamma", gamma, h, d, dev)
    ppg = None if post_gamma is None else _arg("post_gamma", post_gamma, h, d, dev)
    ppb = None if post_beta is None else _arg("post_beta", post_beta, h, d, dev)
    pgt, ng = (None, 1) if gate is None else _gate(gate, M, H, d, dev)
    pdr = None if dresidual is None else _arg("dresidual", dresidual, mh, r, dev)
    pdy = None if dy is None else _arg("dy", dy, mh, d, dev)
    pdga = None if dgamma is None else _arg("dgamma", dgamma, h, _F32, dev)
    pdb = None if dbeta is None else _arg("dbeta", dbeta, h, _F32, dev)
    pdpg = None if dpost_gamma is None else _arg("dpost_gamma", dpost_gamma, h, _F32, dev)
    pdpb = None if dpost_beta is None else _arg("dpost_beta", dpost_beta, h, _F32, dev)
    pdg = None if dgate is None else _arg("dgate", dgate, (H,) if gate is not None and gate.dim() == 1 else (ng, H),
                                          _F32, dev)
    n = _sized_by("te_residual_norm_bwd_workspace", M, H, ng) if workspace is None else 0
    workspace, pw, nw = _workspace_of(n, dout, workspace, stream)
    st = lib().te_residual_norm_bwd(pd, pxo, px, py, _dt(dout), _dt(x_out), M, H, pm, prs, ppm, pprs, pg, ppg, ppb,
                                    pgt, ng, float(residual_scale), _norm_id(norm_type),
                                    int(bool(zero_centered_gamma)), pdr, pdy, pdga, pdb, pdpg, pdpb, pdg, pw, nw,
                                    _stream(stream, dev))
    _check("te_residual_norm_bwd", st)


def te_dense_residual_fwd(x, kernel, residual, out, bias=None, activation="identity", gate=None, residual_scale=1.0,
                          saved_z=None, x_scale_inv=None, kernel_scale_inv=None, workspace=None, stream=None):
    """out = residual_scale * residual + gate * act(x @ kernel + bias); x [M, K] and kernel [K, N] bfloat16 or
    E4M3, bias and gate ([N] or [G, N]) bfloat16.  out may be residual; saved_z [M, N] bfloat16 receives
    x @ kernel + bias."""
    M, K = x.shape
    N = kernel.shape[1]
    dev = torch.cuda.current_device()
    bf = _BF16
    e4m3 = x.dtype in _E4M3_BYTES
    px = _arg("x", x, (M, K), _GEMM_DTYPES, dev)
    pk = _arg("kernel", kernel, (K, N), _E4M3_BYTES if e4m3 else bf, dev)
    pr = _arg("residual", residual, (M, N), _ACT_DTYPES, dev)
    po = _arg("out", out, (M, N), (residual.dtype,), dev)
    pb = None if bias is None else _arg("bias", bias, (N,), bf, dev)
    pz = None if saved_z is None else _arg("saved_z", saved_z, (M, N), bf, dev)
    pgt, ng = (None, 1) if gate is None else _gate(gate, M, N, bf, dev)
    n = _sized_by("te_dense_residual_fwd_workspace", M, K, N, _dt(x)) if workspace is None else 0
    pw, nw = None, 0
    if n or workspace is not None:
        workspace, pw, nw = _workspace_of(n, x, workspace, stream)
    st = lib().te_dense_residual_fwd(px, pk, _dt(x), _scalar("x_scale_inv", x_scale_inv, dev),
                                     _scalar("kernel_scale_inv", kernel_scale_inv, dev), pb, _act_id(activation), pgt,
                                     ng, pr, _dt(residual), float(residual_scale), M, K, N, po, pz, pw, nw,
                                     _stream(stream, dev))
    _check("te_dense_residual_fwd", st)
    return out


def te_dense_residual_bwd(dout, x, kernel, dx, dkernel, dresidual=None, saved_z=None, activation="identity", gate=None,
                          residual_scale=1.0, dbias=None, dgate=None, q=None, x_scale_inv=None, kernel_scale_inv=None,
                          workspace=None, stream=None):
    """Gradients of te_dense_residual_fwd from dout [M, N]; q: the quantizer of dz with E4M3 operands."""
    M, K = x.shape
    N = kernel.shape[1]
    dev = torch.cuda.current_device()
    bf = _BF16
    e4m3 = x.dtype in _E4M3_BYTES
    px = _arg("x", x, (M, K), _GEMM_DTYPES, dev)
    pk = _arg("kernel", kernel, (K, N), _E4M3_BYTES if e4m3 else bf, dev)
    pd = _arg("dout", dout, (M, N), _ACT_DTYPES, dev)
    pz = None if saved_z is None else _arg("saved_z", saved_z, (M, N), bf, dev)
    pgt, ng = (None, 1) if gate is None else _gate(gate, M, N, bf, dev)
    pdx, pdk = _arg("dx", dx, (M, K), bf, dev), _arg("dkernel", dkernel, (K, N), bf, dev)
    pdr = None if dresidual is None else _arg("dresidual", dresidual, (M, N), (dout.dtype,), dev)
    pdb = None if dbias is None else _arg("dbias", dbias, (N,), _F32, dev)
    pdg = None if dgate is None else _arg("dgate", dgate, (N,) if gate is not None and gate.dim() == 1 else (ng, N),
                                          _F32, dev)
    cq = None if q is None else ctypes.byref(_quantizer("q", q, dev))
    n = _sized_by("te_dense_residual_bwd_workspace", M, K, N, ng, _dt(x)) if workspace is None else 0
    workspace, pw, nw = _workspace_of(n, x, workspace, stream)
    st = lib().te_dense_residual_bwd(pd, _dt(dout), px, pk, _dt(x), pz, _act_id(activation), pgt, ng,
                                     float(residual_scale), cq, _scalar("x_scale_inv", x_scale_inv, dev),
                                     _scalar("kernel_scale_inv", kernel_scale_inv, dev), M, K, N, pdx, pdk, pdr, pdb,
                                     pdg, pw, nw, _stream(stream, dev))
    _check("te_dense_residual_bwd", st)
    return dx


class GradList:
    """Gradients for te_grad_norm and te_clip_grad_norm: dense float32 / bfloat16 tensors on one device, and
    outs, where their clipped values go (None: in place).  It keeps the tensors; where they lie, their sizes
    and types are read at each call, so that a tensor may change them in between (resize_, a new .data)."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        self.device = self._table()[1]

    def _table(self):
        """The C table, and the index of its device (-1 the CPU, None of an empty list)."""
        n = len(self.grads)
        if self.outs is not None and len(self.outs) != n:
            raise ValueError("outs: one for each gradient")
        if _read_grads is None:
            lib()
        table, dev = (_Grad * max(n, 1))(), _i64(-1)  # a call's own: another thread may use the list
        i = _read_grads(self.grads, self.outs, n, table, dev)
        if i >= 0:
            self._refuse(i, n)
        return table, dev.value if n else None

    def _refuse(self, i, n):
        if i == n:
            raise ValueError("grads and outs: lists, which keep their length during a call")
        g, dev = self.grads[i], self.grads[0].get_device()
        _arg("grads", g, g.shape, _ACT_DTYPES, dev)
        if self.outs is not None:
            _arg("outs", self.outs[i], g.shape, (g.dtype,), dev)
        raise ValueError(f"grads: entry {i} is not a dense float32 or bfloat16 tensor")


def _grad_args(grads, norm, outs, workspace, stream):
    if not isinstance(grads, GradList):
        grads = GradList(grads, outs)
    elif outs is not None:
        raise ValueError("outs: given with the GradList")
    table, where = grads._table()
    dev = torch.cuda.current_device()
    if where is not None and where != dev:
        raise ValueError(f"grads: tensors must live on the current device (cuda:{dev})")
    pn = _arg("norm", norm.reshape(-1), (1,), _F32, dev)
    n = len(grads.grads)
    size = _sized_by("te_grad_norm_workspace", n) if workspace is None else 0
    workspace, pw, nw = _workspace_of(size, norm, workspace, stream)
    return table, n, pn, workspace, pw, nw, _stream(stream, dev)


def te_grad_norm(grads, norm, workspace=None, stream=None):
    """norm (one float32) = the root of the sum of the squares of all values of the tensors `grads` (a list, or
    a GradList)."""
    table, n, pn, workspace, pw, nw, s = _grad_args(grads, norm, None, workspace, stream)
    _check("te_grad_norm", lib().te_grad_norm(table, n, pn, pw, nw, s))
    return norm


def te_clip_grad_norm(grads, max_norm, norm, outs=None, epsilon=1e-6, workspace=None, stream=None):
    """te_grad_norm, and every value times min(1, max_norm / (norm + epsilon)): in place, or into outs."""
    table, n, pn, workspace, pw, nw, s = _grad_args(grads, norm, outs, workspace, stream)
    _check("te_clip_grad_norm", lib().te_clip_grad_norm(table, n, float(max_norm), float(epsilon), pn, pw, nw, s))
    return norm

"""The block-scaled entry points refuse bad arguments on the host, before any CUDA call (aligned
stand-in addresses that nothing reads), and size their buffers (CPU only)."""

import ctypes
import threading

import pytest
import torch

import fp8_transformer_gb300 as te

b = te.binding
P = 4096
ODD = P + 8  # misaligned


def quantizer(mode=b.TE_SCALING_DELAYED, scale=P, inv=P, amax=P):
    return ctypes.byref(b._Quantizer(scale, inv, amax, mode))


def test_scale_bytes():
    assert te.block_scale_bytes("mxfp4", 1, 32) == 512
    assert te.block_scale_bytes("mxfp4", 129, 160) == 2 * 2 * 512
    assert te.block_scale_bytes("nvfp4", 128, 64) == 512
    assert te.block_scale_bytes("nvfp4", 128, 96) == 1024
    assert te.block_scale_bytes("mxfp8", 0, 64) == 0
    assert te.lib().te_block_scale_bytes(9, 128, 64) == 0
    assert te.lib().te_block_scale_bytes(b.TE_MXFP4, -1, 64) == 0
    # past 32 bits
    assert te.block_scale_bytes("nvfp4", 1 << 22, 1 << 16) == (1 << 22) * (1 << 12)


def test_workspace_sizes():
    ws = te.workspace_size(b.TE_OP_DENSE_FP4_FWD, 33, 4096, 512)
    assert ws >= 33 * 2048 + te.block_scale_bytes("nvfp4", 33, 4096)
    ws = te.workspace_size(b.TE_OP_DENSE_FP4_BWD, 33, 4096, 512)
    assert ws >= 33 * 256 + 512 * 32 + te.block_scale_bytes("nvfp4", 33, 512) + te.block_scale_bytes("nvfp4", 512, 64)
    assert te.workspace_size(b.TE_OP_DENSE_FP4_FWD, 0, 4096, 512) == 0


def quantize(x=P, dt=b.TE_BF16, M=4, N=64, f=b.TE_MXFP4, q=None, c=P, s=P, ct=None, st=None):
    return te.lib().te_block_quantize(x, dt, M, N, f, q, c, s, ct, st, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(dt=b.TE_E4M3), dict(M=-1), dict(N=0), dict(f=7), dict(s=None),
                                dict(c=None, s=None), dict(ct=P), dict(q=quantizer()), dict(f=b.TE_NVFP4),
                                dict(f=b.TE_NVFP4, q=quantizer(scale=None)),
                                dict(f=b.TE_NVFP4, q=quantizer(mode=b.TE_SCALING_CURRENT, amax=None)),
                                dict(f=b.TE_NVFP4, q=quantizer(mode=5))])
def test_quantize_invalid(kw):
    assert quantize(**kw) == b.TE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(N=48), dict(N=40, c=None, s=None, ct=P, st=P), dict(x=ODD), dict(c=ODD), dict(s=ODD), dict(ct=ODD, st=P),
                                dict(f=b.TE_MXFP8, ct=P, st=P)])
def test_quantize_unsupported(kw):
    assert quantize(**kw) == b.TE_ERR_UNSUPPORTED


def test_nothing_to_do_without_rows():
    assert quantize(M=0, x=None) == b.TE_OK
    assert te.lib().te_block_dequantize(None, None, b.TE_MXFP4, None, 0, 64, None, b.TE_F32, None) == b.TE_OK
    assert te.lib().te_block_gemm(None, None, P, P, b.TE_MXFP4, 0, 64, 64, None, None, None, b.TE_F32, None,
                                  b.TE_F32, None) == b.TE_OK


def test_dequantize_refusals():
    def f(c=P, s=P, fmt=b.TE_MXFP4, inv=None, M=4, N=64, o=P, dt=b.TE_F32):
        return te.lib().te_block_dequantize(c, s, fmt, inv, M, N, o, dt, None)
    for kw in (dict(c=None), dict(s=None), dict(o=None), dict(fmt=-1), dict(inv=P), dict(dt=b.TE_E4M3), dict(N=-32)):
        assert f(**kw) == b.TE_ERR_INVALID_ARG, kw
    for kw in (dict(N=16), dict(c=ODD), dict(o=ODD), dict(fmt=b.TE_NVFP4, inv=P + 2)):
        assert f(**kw) == b.TE_ERR_UNSUPPORTED, kw


def test_gemm_refusals():
    def f(a=P, fmt=b.TE_MXFP4, M=4, N=64, K=64, ia=None, bias=None, bdt=b.TE_F32, D=P, ddt=b.TE_BF16):
        return te.lib().te_block_gemm(a, P, P, P, fmt, M, N, K, ia, None, bias, bdt, D, ddt, None)
    for kw in (dict(a=None), dict(D=None), dict(M=-1), dict(K=0), dict(N=0), dict(ddt=b.TE_E4M3), dict(fmt=3),
               dict(bias=P, bdt=b.TE_E4M3)):
        assert f(**kw) == b.TE_ERR_INVALID_ARG, kw
    for kw in (dict(fmt=b.TE_MXFP8), dict(N=24), dict(K=48), dict(a=ODD), dict(bias=ODD), dict(ia=P + 1),
               dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 16), dict(K=1 << 31)):
        assert f(**kw) == b.TE_ERR_UNSUPPORTED, kw


def test_dense_refusals():
    big = 1 << 30

    def fwd(x=P, dt=b.TE_BF16, fmt=b.TE_MXFP4, q=None, M=4, K=64, N=64, xt=None, xts=None, ws=P, n=big):
        return te.lib().te_dense_fp4_fwd(x, dt, P, P, fmt, q, None, None, M, K, N, P, xt, xts, ws, n, None)
    for kw in (dict(x=None), dict(dt=b.TE_E4M3), dict(fmt=b.TE_NVFP4), dict(q=quantizer()), dict(xt=P),
               dict(fmt=b.TE_NVFP4, q=quantizer(inv=None)), dict(K=-64)):
        assert fwd(**kw) == b.TE_ERR_INVALID_ARG, kw
    for kw in (dict(fmt=b.TE_MXFP8), dict(K=48), dict(N=24), dict(x=ODD), dict(xt=ODD, xts=P), dict(ws=ODD)):
        assert fwd(**kw) == b.TE_ERR_UNSUPPORTED, kw
    assert fwd(M=9, ws=None) == b.TE_ERR_WORKSPACE and fwd(M=9, n=100) == b.TE_ERR_WORKSPACE
    assert fwd(xt=P, xts=P, ws=None) == b.TE_ERR_WORKSPACE
    assert fwd(M=0) == b.TE_OK
    # the call's own factor in the place of the kernel's
    assert te.lib().te_dense_fp4_fwd(P, b.TE_BF16, P, P, b.TE_NVFP4, quantizer(inv=P + 64), P + 64, None, 4, 64, 64, P, None,
                                     None, P, big, None) == b.TE_ERR_INVALID_ARG

    def bwd(dy=P, dw=P, fmt=b.TE_MXFP4, q=None, M=4, K=64, N=64, db=None, ws=P, n=big):
        return te.lib().te_dense_fp4_bwd(dy, b.TE_BF16, P, P, P, P, fmt, q, None, None, M, K, N, P, dw, db, ws, n, None)
    for kw in (dict(dy=None), dict(dw=None), dict(fmt=b.TE_NVFP4), dict(q=quantizer()), dict(N=0)):
        assert bwd(**kw) == b.TE_ERR_INVALID_ARG, kw
    for kw in (dict(fmt=b.TE_MXFP8), dict(N=80), dict(K=16), dict(dy=ODD), dict(db=P + 2)):
        assert bwd(**kw) == b.TE_ERR_UNSUPPORTED, kw
    for fac in ((P + 64, None), (None, P + 64)):
        assert te.lib().te_dense_fp4_bwd(P, b.TE_BF16, P, P, P, P, b.TE_NVFP4, quantizer(inv=P + 64), *fac, 4, 64, 64, P, P,
                                         None, P, big, None) == b.TE_ERR_INVALID_ARG
    assert bwd(ws=None) == b.TE_ERR_WORKSPACE and bwd(n=100) == b.TE_ERR_WORKSPACE


def test_checkpoint_refusals():
    def f(dy=P, s=P, dt=b.TE_BF16, N=64, act=b.TE_GELU, q=None, dx=P, dxt=b.TE_BF16, a=None, db=None, ws=None, n=0):
        return te.lib().te_dact_dbias_ckpt(dy, P, s, dt, 4, N, act, q, dx, dxt, a, db, ws, n, None)
    for kw in (dict(dy=None), dict(s=None), dict(dx=None), dict(act=b.TE_IDENTITY), dict(act=12), dict(dt=b.TE_E4M3),
               dict(dxt=b.TE_E4M3), dict(q=quantizer(mode=9))):
        assert f(**kw) == b.TE_ERR_INVALID_ARG, kw
    for kw in (dict(N=48), dict(act=b.TE_SWIGLU, N=96), dict(dy=ODD), dict(a=ODD), dict(db=P + 2, ws=P, n=1 << 20),
               dict(db=P, ws=ODD, n=1 << 20)):
        assert f(**kw) == b.TE_ERR_UNSUPPORTED, kw
    assert f(db=P) == b.TE_ERR_WORKSPACE and f(db=P, ws=P, n=16) == b.TE_ERR_WORKSPACE


def test_the_bindings_scale_size_is_the_librarys():
    for f in range(3):
        for rows in (0, 1, 127, 128, 129, 1000):
            for cols in (32, 64, 96, 128, 160, 4096):
                assert b._scale_size(f, rows, cols) == te.lib().te_block_scale_bytes(f, rows, cols)


@pytest.mark.parametrize("q,ok", [(dict(), False), (dict(inv=P + 64), False), (dict(inv=P + 64, amax=P + 128), True),
                                  (dict(inv=P + 64, amax=P + 128, mode=b.TE_SCALING_CURRENT), False)])
def test_a_factor_that_the_call_would_write(q, ok):
    """The kernel's factor at P in a quantizer's own places (scale at P by default): refused where the call writes
    there; a delayed scale is only read.  Valid calls are stopped by their missing workspace."""
    want = b.TE_ERR_WORKSPACE if ok else b.TE_ERR_INVALID_ARG
    for k, x in ((P, None), (None, P)):
        assert te.lib().te_dense_fp4_bwd(P, b.TE_BF16, P, P, P, P, b.TE_NVFP4, quantizer(**q), k, x, 4, 64, 64, P, P,
                                         None, None, 0, None) == want
    assert te.lib().te_dense_fp4_fwd(P, b.TE_BF16, P, P, b.TE_NVFP4, quantizer(**q), P, None, 16, 64, 64, P, None,
                                     None, None, 0, None) == want


def test_a_callers_workspace_is_counted_in_bytes_and_is_dense():
    w = torch.empty(100, dtype=torch.float32)
    assert b._given_workspace(w, -1) == (w.data_ptr(), 400)
    assert b._given_workspace(w[10:20], -1) == (w.data_ptr() + 40, 40)
    for bad, dev in ((w[::2], -1), (w[:1].expand(1 << 20), -1), (w, 0)):
        with pytest.raises(ValueError, match="workspace"):
            b._given_workspace(bad, dev)


def test_workspaces_are_kept_for_torchs_own_streams_alone(monkeypatch):
    """A stream made elsewhere may be destroyed and its handle come back: its calls get a buffer each."""
    now = {}
    monkeypatch.setattr(b, "_raw_stream", lambda dev: now["handle"])
    monkeypatch.setattr(b, "_stream_data", lambda dev: (now["id"], 0, 1))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now.get("capturing", False))
    monkeypatch.setattr(b, "_small", threading.local())
    like = torch.empty(1)

    def take(sid, handle, **kw):
        now.update(id=sid, handle=handle, **kw)
        return b._workspace(b.TE_OP_DENSE_FP4_FWD, 9, 64, 64, like, None, None)
    default, pooled = take(0, 0), take(35, 0x5000)
    assert take(0, 0)[1] == default[1] and take(35, 0x5000)[1] == pooled[1] != default[1]
    assert default[2] == pooled[2] == 1 << 20
    first, second = take(0x7000, 0x7000), take(0x7000, 0x7000)
    assert first[1] != second[1] and first[2] == te.workspace_size(b.TE_OP_DENSE_FP4_FWD, 9, 64, 64)
    assert take(35, 0x5000, capturing=True)[1] != pooled[1]
    assert sorted(b._small.kept) == [(-1, 0), (-1, 0x5000)]

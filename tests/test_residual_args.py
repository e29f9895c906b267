"""The entry points around the residual stream refuse bad arguments on the host, before any CUDA call
(aligned stand-in addresses that nothing reads; CPU only)."""

import ctypes

import pytest
import torch

import fp8_transformer_gb300 as te

b = te.binding
MB = 1 << 20
P = {k: (i + 1) * 64 * MB for i, k in enumerate(
    "y residual gamma beta post_gamma post_beta gate x_out out mu rsigma post_mu post_rsigma dout dx_out dresidual dy dgamma "
    "dbeta dpost_gamma dpost_beta dgate ws x kernel bias z dx dkernel dbias scale scale_inv amax xs ks".split())}


def quantizer(mode=b.TE_SCALING_DELAYED, **kw):
    return ctypes.byref(b._Quantizer(kw.get("scale", P["scale"]), kw.get("inv", P["scale_inv"]), kw.get("amax", P["amax"]), mode))


def fwd(dtype=b.TE_BF16, rtype=b.TE_BF16, M=4, H=64, gates=2, norm=b.TE_LAYERNORM, q=None, od=b.TE_BF16, **kw):
    a = {**P, **kw}
    return te.lib().te_residual_norm_fwd(a["y"], dtype, a["residual"], rtype, M, H, a["gamma"], a["beta"], a["post_gamma"],
                                         a["post_beta"], a["gate"], gates, 1.0, norm, 0, 1e-6, q, a["x_out"], a["out"], od,
                                         a["mu"], a["rsigma"], a["post_mu"], a["post_rsigma"], None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(residual=None), dict(gamma=None), dict(x_out=None), dict(out=None), dict(M=-1), dict(H=0),
    dict(dtype=b.TE_E4M3), dict(dtype=b.TE_F32), dict(rtype=b.TE_E4M3), dict(norm=7), dict(od=5), dict(od=b.TE_E4M3),
    dict(gates=0), dict(gates=3), dict(gates=-2), dict(post_gamma=None), dict(od=b.TE_E4M3, q=quantizer(mode=4)),
    dict(od=b.TE_E4M3, q=quantizer(b.TE_SCALING_CURRENT, amax=None)),
    # what is written overlaps something
    dict(x_out=P["y"]), dict(x_out=P["residual"] + 16), dict(out=P["residual"]), dict(out=P["x_out"]), dict(out=P["gamma"]),
    dict(mu=P["rsigma"]), dict(out=P["gate"] + 128), dict(od=b.TE_E4M3, q=quantizer(amax=P["mu"])),
    dict(od=b.TE_E4M3, q=quantizer(inv=P["out"]))])
def test_norm_fwd_invalid(kw):
    assert fwd(**kw) == b.TE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(H=60), dict(H=8200), dict(y=P["y"] + 8), dict(gate=P["gate"] + 2), dict(mu=P["mu"] + 2),
                                dict(out=P["out"] + 4), dict(M=(1 << 30) + 2)])
def test_norm_fwd_unsupported(kw):
    assert fwd(**kw) == b.TE_ERR_UNSUPPORTED


def bwd(dtype=b.TE_BF16, rtype=b.TE_BF16, M=4, H=64, gates=2, norm=b.TE_LAYERNORM, n=64 * MB, **kw):
    a = {**P, **kw}
    return te.lib().te_residual_norm_bwd(a["dout"], a["dx_out"], a["x_out"], a["y"], dtype, rtype, M, H, a["mu"], a["rsigma"],
                                         a["post_mu"], a["post_rsigma"], a["gamma"], a["post_gamma"], a["post_beta"],
                                         a["gate"], gates, 1.0, norm, 0, a["dresidual"], a["dy"], a["dgamma"], a["dbeta"],
                                         a["dpost_gamma"], a["dpost_beta"], a["dgate"], a["ws"], n, None)


@pytest.mark.parametrize("kw", [
    dict(dout=None), dict(x_out=None), dict(mu=None), dict(rsigma=None), dict(gamma=None), dict(dgamma=None), dict(y=None),
    dict(post_mu=None), dict(post_rsigma=None), dict(post_gamma=None), dict(gate=None), dict(gates=3), dict(gates=0),
    dict(dtype=b.TE_F32), dict(M=-1), dict(H=0), dict(norm=2), dict(dy=P["dout"]), dict(dresidual=P["dx_out"] + 16),
    dict(dgamma=P["dbeta"]), dict(dgate=P["ws"]), dict(ws=P["dy"]), dict(dresidual=P["x_out"])])
def test_norm_bwd_invalid(kw):
    assert bwd(**kw) == b.TE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(H=68), dict(H=9000), dict(dout=P["dout"] + 8), dict(dgate=P["dgate"] + 2), dict(ws=P["ws"] + 4),
                                dict(M=(1 << 30) + 2)])
def test_norm_bwd_unsupported(kw):
    assert bwd(**kw) == b.TE_ERR_UNSUPPORTED


def test_norm_bwd_workspace():
    assert bwd(ws=None) == b.TE_ERR_WORKSPACE and bwd(n=64) == b.TE_ERR_WORKSPACE
    f = te.lib().te_residual_norm_bwd_workspace
    assert f(0, 64, 1) == 0 and f(4, 0, 1) == 0
    assert f(4, 64, 2) >= (4 + 4 + 2) * 2 * 64 * 4 // 4
    assert f(1 << 20, 8192, 1 << 20) > 1 << 36  # past 32 bits


def dense(dtype=b.TE_BF16, rtype=b.TE_BF16, act=b.TE_GELU, gates=2, M=4, K=64, N=64, n=64 * MB, **kw):
    a = {**P, "xs": None, "ks": None, **kw}
    return te.lib().te_dense_residual_fwd(a["x"], a["kernel"], dtype, a["xs"], a["ks"], a["bias"], act, a["gate"], gates,
                                          a["residual"], rtype, 1.0, M, K, N, a["out"], a["z"], a["ws"], n, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(kernel=None), dict(residual=None), dict(out=None), dict(dtype=b.TE_F32), dict(rtype=b.TE_E4M3),
    dict(act=b.TE_SWIGLU), dict(act=-1), dict(gates=3), dict(gates=0), dict(M=-1), dict(K=0), dict(N=0), dict(xs=P["xs"]),
    dict(out=P["residual"] + 32), dict(out=P["x"]), dict(out=P["kernel"] + 64), dict(z=P["out"]), dict(z=P["residual"]),
    dict(z=P["bias"]), dict(out=P["gate"])])
def test_dense_fwd_invalid(kw):
    assert dense(**kw) == b.TE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(K=72), dict(N=40), dict(x=P["x"] + 8), dict(bias=P["bias"] + 2), dict(gate=P["gate"] + 8),
                                dict(dtype=b.TE_E4M3, xs=P["xs"] + 1), dict(M=(1 << 30) + 2), dict(K=(1 << 30) + 16),
                                dict(N=1 << 31), dict(ws=P["ws"] + 8)])
def test_dense_fwd_unsupported(kw):
    assert dense(**kw) == b.TE_ERR_UNSUPPORTED


def dense_bwd(dtype=b.TE_BF16, rtype=b.TE_BF16, act=b.TE_GELU, gates=2, M=4, K=64, N=64, q=None, n=64 * MB, **kw):
    a = {**P, "xs": None, "ks": None, **kw}
    return te.lib().te_dense_residual_bwd(a["dout"], rtype, a["x"], a["kernel"], dtype, a["z"], act, a["gate"], gates, 1.0, q,
                                          a["xs"], a["ks"], M, K, N, a["dx"], a["dkernel"], a["dresidual"], a["dbias"],
                                          a["dgate"], a["ws"], n, None)


@pytest.mark.parametrize("kw", [
    dict(dout=None), dict(x=None), dict(kernel=None), dict(dx=None), dict(dkernel=None), dict(z=None), dict(gate=None),
    dict(act=b.TE_IDENTITY, z=None), dict(q=quantizer()), dict(dtype=b.TE_E4M3), dict(dtype=b.TE_E4M3, q=quantizer(inv=None)),
    dict(dtype=b.TE_E4M3, q=quantizer(inv=P["xs"]), xs=P["xs"]), dict(dtype=b.TE_E4M3, q=quantizer(amax=P["ks"]), ks=P["ks"]),
    dict(dtype=b.TE_F32), dict(act=b.TE_GEGLU), dict(gates=3), dict(dresidual=P["dout"]), dict(dx=P["x"]),
    dict(dkernel=P["kernel"]), dict(dbias=P["dgate"]), dict(ws=P["dx"]), dict(xs=P["xs"]), dict(M=-4)])
def test_dense_bwd_invalid(kw):
    assert dense_bwd(**kw) == b.TE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(K=72), dict(N=40), dict(dout=P["dout"] + 8), dict(dbias=P["dbias"] + 2), dict(M=(1 << 30) + 2)])
def test_dense_bwd_unsupported(kw):
    assert dense_bwd(**kw) == b.TE_ERR_UNSUPPORTED


def test_dense_bwd_workspace():
    assert dense_bwd(ws=None) == b.TE_ERR_WORKSPACE and dense_bwd(n=128) == b.TE_ERR_WORKSPACE


NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would go on to the launch")


@NO_GPU
def test_what_is_not_read_is_not_held_against_what_is_written():
    """Tensors that a call takes and does not read may lie anywhere (these pass the checks and find no device)."""
    rms, plain = b.TE_RMSNORM, dict(post_gamma=None, post_beta=None, post_mu=None, post_rsigma=None)
    for kw in (dict(norm=rms, beta=P["out"]), dict(norm=rms, post_beta=P["x_out"] + 8),
               dict(q=quantizer(scale=P["out"], inv=P["x_out"]))):
        assert fwd(**kw) == b.TE_ERR_CUDA, kw
    assert fwd(q=quantizer(amax=P["out"])) == b.TE_ERR_INVALID_ARG
    assert fwd(od=b.TE_E4M3, q=quantizer(scale=P["out"])) == b.TE_ERR_INVALID_ARG
    none = dict(plain, gate=None, dgate=None, dpost_gamma=None, dpost_beta=None)
    for kw in (dict(none, dy=P["y"]), dict(none, y=P["dresidual"] + 8), dict(norm=rms, mu=P["dy"]),
               dict(norm=rms, post_mu=P["dgamma"] + 1), dict(norm=rms, post_beta=P["dy"]),
               dict(post_beta=P["dy"], dgate=None)):
        assert bwd(**kw) == b.TE_ERR_CUDA, kw
    for kw in (dict(dy=P["y"]), dict(none, dy=P["x_out"]), dict(norm=rms, rsigma=P["dy"]), dict(post_beta=P["dy"])):
        assert bwd(**kw) == b.TE_ERR_INVALID_ARG, kw
    for kw in (dict(act=b.TE_IDENTITY, dgate=None, z=P["dx"]), dict(act=b.TE_IDENTITY, dgate=None, z=P["dbias"] + 2)):
        assert dense_bwd(**kw) == b.TE_ERR_CUDA, kw
    for kw in (dict(act=b.TE_IDENTITY, z=P["dx"]), dict(act=b.TE_RELU, dgate=None, z=P["dx"])):
        assert dense_bwd(**kw) == b.TE_ERR_INVALID_ARG, kw


@NO_GPU
def test_dense_bwd_many_columns():
    """More than 65535 strips of 256 columns pass the checks (and find no device here)."""
    far = {k: (i + 1) << 40 for i, k in enumerate(P)}
    kw = dict(far, dtype=b.TE_E4M3, q=quantizer(scale=far["scale"], inv=far["scale_inv"], amax=None), M=2, K=16, n=1 << 34)
    for N in (65535 * 256, 65535 * 256 + 16, 1 << 28):
        assert dense_bwd(N=N, **kw) == b.TE_ERR_CUDA, N


def grads(*spec):
    return (b._Grad * max(len(spec), 1))(*(b._Grad(*s) for s in spec))


def clip(spec, max_norm=1.0, eps=1e-6, norm=P["amax"], ws=P["ws"], n=64 * MB, count=None):
    return te.lib().te_clip_grad_norm(grads(*spec), len(spec) if count is None else count, max_norm, eps, norm, ws, n, None)


def test_clip_refusals():
    ok = (P["x"], None, 100, b.TE_F32)
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")), dict(eps=-1e-6),
               dict(eps=float("nan")), dict(norm=None), dict(count=-1)):
        assert clip([ok], **kw) == b.TE_ERR_INVALID_ARG, kw
    for bad in ((None, None, 5, b.TE_F32), (P["x"], None, -1, b.TE_F32), (P["x"], None, 5, b.TE_E4M3), (P["x"], None, 5, 9)):
        assert clip([ok if bad[0] else bad, bad]) == b.TE_ERR_INVALID_ARG, bad
    X, Y = P["x"], P["y"]
    for spec in ([ok, ok], [ok, (X + 396, None, 4, b.TE_F32)], [ok, (Y, X + 4, 10, b.TE_F32)], [(X, X + 4, 10, b.TE_F32)],
                 [(X, Y, 10, b.TE_F32), (X, None, 10, b.TE_F32)], [(X, Y, 10, b.TE_F32), (Y + 36, P["z"], 10, b.TE_F32)],
                 [(P["amax"] - 8, None, 3, b.TE_F32)], [(P["amax"] - 8, Y, 3, b.TE_F32)]):
        assert clip(spec) == b.TE_ERR_INVALID_ARG, spec
    for bad in ((X + 2, None, 5, b.TE_F32), (X + 1, None, 5, b.TE_BF16), (X, Y + 1, 5, b.TE_BF16)):
        assert clip([bad]) == b.TE_ERR_UNSUPPORTED, bad
    assert clip([ok], norm=P["amax"] + 1) == b.TE_ERR_UNSUPPORTED
    assert clip([ok], ws=P["ws"] + 8) == b.TE_ERR_UNSUPPORTED
    assert clip([ok], ws=None) == b.TE_ERR_WORKSPACE and clip([ok], n=4) == b.TE_ERR_WORKSPACE


@pytest.mark.parametrize("call", ["te_grad_norm", "te_clip_grad_norm"])
def test_gradients_workspace_overlaps_nothing(call):
    """The workspace on a gradient, on the place of a clipped one, on the norm, and beside them."""
    lib, W, X = te.lib(), P["ws"], P["x"]
    n = lib.te_grad_norm_workspace(1)
    assert n >= 16

    def run(spec, ws=W, norm=P["amax"], nbytes=64 * MB):
        mid = (1.0, 1e-6) if call == "te_clip_grad_norm" else ()
        return getattr(lib, call)(grads(spec), 1, *mid, norm, ws, nbytes, None)

    inside = [W, W + n - 4, W - 396]
    for at in inside:
        assert run((at, None, 100, b.TE_F32)) == b.TE_ERR_INVALID_ARG, at
    for at in (W, W + 4, W + n - 4):
        assert run((X, None, 100, b.TE_F32), norm=at) == b.TE_ERR_INVALID_ARG, at
    if call == "te_clip_grad_norm":
        for at in inside:
            assert run((X, at, 100, b.TE_F32)) == b.TE_ERR_INVALID_ARG, at
    # a workspace that is too short is refused for that, unless what there is of it overlaps already
    assert run((X, None, 100, b.TE_F32), nbytes=n - 1) == b.TE_ERR_WORKSPACE
    assert run((W, None, 100, b.TE_F32), nbytes=n - 1) == b.TE_ERR_INVALID_ARG
    # (neighbours are allowed: these go on to the launch, which finds no device here or is not made)
    if not torch.cuda.is_available():
        for spec in ((W + n, None, 100, b.TE_F32), (W - 400, None, 100, b.TE_F32)):
            assert run(spec) == b.TE_ERR_CUDA, spec
        assert run((X, None, 100, b.TE_F32), norm=W + n) == b.TE_ERR_CUDA


def test_binding_refuses_cpu_tensors_and_shapes():
    lst = te.GradList([torch.ones(3)])
    assert lst.device == -1
    with pytest.raises(ValueError):
        te.GradList([torch.ones(3), torch.ones(3).double()])
    with pytest.raises(ValueError):
        te.GradList([torch.ones(4, 4).t()[:2]])
    with pytest.raises(ValueError):
        te.GradList([torch.ones(3)], [])
    with pytest.raises(ValueError):
        te.GradList([torch.ones(3)], [torch.ones(4)])
    with pytest.raises(ValueError):
        b._gate(torch.ones(3, 8), 4, 8, (torch.float32,), -1)

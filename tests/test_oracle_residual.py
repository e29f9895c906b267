"""Pins of oracle/residual.py: differences of its own forward passes, and torch's float64 autograd (CPU)."""

import numpy as np
import pytest
import torch

from oracle import residual as rs


def _norm(x, gamma, beta, ln, zc, eps):
    g = gamma + 1 if zc else gamma
    if ln:
        return torch.nn.functional.layer_norm(x, x.shape[-1:], g, beta, eps)
    return torch.nn.functional.rms_norm(x, x.shape[-1:], g, eps)


@pytest.mark.parametrize("ln", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("G", [0, 1, 3])
def test_residual_norm_against_autograd(ln, post, G):
    g = torch.Generator().manual_seed(5)
    M, H, eps, scale, zc = 6, 16, 1e-5, 0.7, True
    t = {k: torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True) for k, s in
         dict(y=(M, H), residual=(M, H), gamma=(H,), beta=(H,), post_gamma=(H,), post_beta=(H,),
              gate=(max(G, 1), H)).items()}
    p = _norm(t["y"], t["post_gamma"], t["post_beta"], ln, zc, eps) if post else t["y"]
    gate = t["gate"].repeat_interleave(M // max(G, 1), 0) if G else 1.0
    x = scale * t["residual"] + gate * p
    out = _norm(x, t["gamma"], t["beta"], ln, zc, eps)
    dout, dxo = torch.randn(M, H, generator=g, dtype=torch.float64), torch.randn(M, H, generator=g, dtype=torch.float64)
    ((out * dout).sum() + (x * dxo).sum()).backward()
    n = {k: v.detach().numpy() for k, v in t.items()}
    kw = dict(post_gamma=n["post_gamma"] if post else None, post_beta=n["post_beta"] if post else None,
              gate=n["gate"] if G else None, scale=scale, layernorm=ln, zc=zc)
    f = rs.residual_norm_fwd(n["y"], n["residual"], n["gamma"], n["beta"], eps=eps, **kw)
    assert np.allclose(f["x_out"][0], x.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(f["out"][0], out.detach().numpy(), rtol=1e-11, atol=1e-11)
    b = rs.residual_norm_bwd(dout.numpy(), dxo.numpy(), f["x_out"][0], f["mu"], f["rsigma"], n["gamma"], y=n["y"],
                             post_mu=f.get("post_mu"), post_rs=f.get("post_rsigma"), **kw)
    want = dict(dresidual="residual", dy="y", dgamma="gamma")
    if ln:
        want["dbeta"] = "beta"
    if post:
        want["dpost_gamma"] = "post_gamma"
        if ln:
            want["dpost_beta"] = "post_beta"
    if G:
        want["dgate"] = "gate"
    for k, leaf in want.items():
        assert np.allclose(b[k][0], t[leaf].grad.numpy(), rtol=1e-10, atol=1e-10), k


@pytest.mark.parametrize("name", ["identity", "relu", "gelu", "silu"])
@pytest.mark.parametrize("G", [0, 1, 2])
def test_dense_residual_against_differences(name, G):
    r = np.random.default_rng(3)
    M, K, N, scale = 4, 6, 5, 0.3
    x, w, res, b = r.normal(size=(M, K)), r.normal(size=(K, N)), r.normal(size=(M, N)), r.normal(size=N)
    gate = r.normal(size=(G, N)) if G else None
    dout = r.normal(size=(M, N))
    z = rs.dense_residual_fwd(x, w, res, b, name, gate, scale)[1]
    e = rs.dense_residual_grad(dout, z, name, gate, scale)
    grads = {"x": e["dz"] @ w.T, "w": x.T @ e["dz"], "res": e["dresidual"], "b": e["dbias"][0]}
    leaves = {"x": x, "w": w, "res": res, "b": b}
    if G:
        grads["gate"], leaves["gate"] = e["dgate"][0], gate
    for k, v in leaves.items():
        for i in np.ndindex(v.shape):
            keep, h = v[i], 1e-6
            f = []
            for s in (h, -h):
                v[i] = keep + s
                f.append((rs.dense_residual_fwd(x, w, res, b, name, gate, scale)[0] * dout).sum())
            v[i] = keep
            assert abs((f[0] - f[1]) / (2 * h) - grads[k][i]) < 1e-6, (k, i)


def test_clip_against_torch():
    g = torch.Generator().manual_seed(0)
    for scale, mx in ((1.0, 0.5), (1.0, 1e6), (0.0, 1.0)):
        ps = [torch.nn.Parameter(torch.zeros(n, dtype=torch.float64)) for n in (1, 17, 40)]
        for p in ps:
            p.grad = torch.randn(p.shape, generator=g, dtype=torch.float64) * scale
        old = [p.grad.numpy().copy() for p in ps]
        n, c = rs.clip(old, mx, 1e-6)
        got = torch.nn.utils.clip_grad_norm_(ps, mx)
        assert abs(n - got.item()) < 1e-12
        for o, p in zip(old, ps):
            assert np.allclose(o * c, p.grad.numpy(), rtol=1e-12)
    assert rs.clip([np.zeros(3)], 1.0, 0.0) == (0.0, 1.0)

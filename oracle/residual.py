"""Oracle of the operators around the residual stream, in float64 numpy (test infrastructure).

Every result comes with the sum of the magnitudes of the terms that form it, which a test's error
window is a multiple of: an fp32 computation of the same terms is off by a few roundings of them.
"""

from __future__ import annotations

import numpy as np

from . import block as ob


def _gain(gamma, zc):
    return gamma + 1.0 if zc else gamma


def gate_rows(gate, M):
    """The gate of each row ([H] or [G, H] -> [M, H]); ones without one."""
    if gate is None:
        return 1.0
    g = np.atleast_2d(gate)
    return np.repeat(g, M // g.shape[0], axis=0)


def norm(x, wx, gamma, beta, layernorm, zc, eps):
    """(values, magnitudes, mu, rsigma); wx: the window of x in units of its rounding (propagated)."""
    mu = x.mean(1, keepdims=True) if layernorm else np.zeros((x.shape[0], 1))
    d = x - mu
    rs = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    g = _gain(gamma, zc)
    b = beta if layernorm and beta is not None else 0.0
    out = d * rs * g + b
    a = np.abs(x) + np.abs(mu)
    # an error e of x moves d by e and its mean, and rs by mean(|d| e) rs^3
    moved = wx + wx.mean(1, keepdims=True) + np.abs(d) * (rs * rs) * (np.abs(d) * wx).mean(1, keepdims=True)
    mag = (a + moved) * rs * np.abs(g) + np.abs(b)
    return out, mag, mu[:, 0], rs[:, 0]


def residual_norm_fwd(y, residual, gamma, beta=None, post_gamma=None, post_beta=None, gate=None, scale=1.0,
                      layernorm=True, zc=False, eps=1e-6):
    """dict of (value, magnitude) for x_out and out, and the statistics."""
    r = {}
    p, w = y, np.abs(y)
    if post_gamma is not None:
        p, w, r["post_mu"], r["post_rsigma"] = norm(y, np.zeros_like(y), post_gamma, post_beta, layernorm, zc, eps)
    g = gate_rows(gate, y.shape[0])
    x = scale * residual + g * p
    wx = np.abs(scale * residual) + np.abs(g) * w
    out, wo, r["mu"], r["rsigma"] = norm(x, wx, gamma, beta, layernorm, zc, eps)
    r["x_out"], r["out"] = (x, wx), (out, wo)
    return r


def _hat(x, mu, rs, layernorm):
    m = mu[:, None] if layernorm else 0.0
    return (x - m) * rs[:, None], (np.abs(x) + np.abs(m)) * rs[:, None]


def _norm_grad(d, wd, h, wh, rs, layernorm):
    """Gradient of a norm's input from the gradient d of its normalized rows, and the magnitudes."""
    g = d - h * (d * h).mean(1, keepdims=True)
    w = wd + wh * (wd * wh).mean(1, keepdims=True)
    if layernorm:
        g = g - d.mean(1, keepdims=True)
        w = w + wd.mean(1, keepdims=True)
    return g * rs[:, None], w * rs[:, None]


def _by_gate(v, gates):
    return v.reshape(gates, -1, v.shape[1]).sum(1)


def residual_norm_bwd(dout, dx_out, x_out, mu, rs, gamma, y=None, post_mu=None, post_rs=None, post_gamma=None,
                      post_beta=None, gate=None, scale=1.0, layernorm=True, zc=False):
    """dict of (value, magnitude) for each gradient."""
    M = dout.shape[0]
    r = {}
    h, wh = _hat(x_out, mu, rs, layernorm)
    g = _gain(gamma, zc)
    dx, wdx = _norm_grad(dout * g, np.abs(dout * g), h, wh, rs, layernorm)
    if dx_out is not None:
        dx, wdx = dx + dx_out, wdx + np.abs(dx_out)
    r["dresidual"] = scale * dx, abs(scale) * wdx
    r["dgamma"] = (dout * h).sum(0), (np.abs(dout) * wh).sum(0)
    r["dbeta"] = (dout.sum(0), np.abs(dout).sum(0)) if layernorm else (np.zeros(dout.shape[1]),) * 2
    gt = gate_rows(gate, M)
    dp, wdp = dx * gt, wdx * np.abs(gt)
    if post_gamma is None:
        ph, wph, p, wp = y, None if y is None else np.abs(y), y, None if y is None else np.abs(y)
        r["dy"] = dp, wdp
    else:
        ph, wph = _hat(y, post_mu, post_rs, layernorm)
        pg = _gain(post_gamma, zc)
        pb = post_beta if layernorm and post_beta is not None else 0.0
        p, wp = ph * pg + pb, wph * np.abs(pg) + np.abs(pb)
        r["dpost_gamma"] = (dp * ph).sum(0), (wdp * wph).sum(0)
        r["dpost_beta"] = (dp.sum(0), wdp.sum(0)) if layernorm else (np.zeros(dout.shape[1]),) * 2
        r["dy"] = _norm_grad(dp * pg, wdp * np.abs(pg), ph, wph, post_rs, layernorm)
    if gate is not None:
        G = np.atleast_2d(gate).shape[0]
        r["dgate"] = _by_gate(dx * p, G), _by_gate(wdx * wp, G)
    return r


def act(name, z):
    """(value, derivative) of an activation."""
    if name == "identity":
        return z, np.ones_like(z)
    return ob.act_fwd(z, name), ob.act_bwd(np.ones_like(z), z, name)


def dense_residual_fwd(x, w, residual, bias=None, name="identity", gate=None, scale=1.0):
    """(out, z, the product's magnitudes)."""
    z = x @ w + (0.0 if bias is None else bias)
    mag = np.abs(x) @ np.abs(w)
    return scale * residual + gate_rows(gate, x.shape[0]) * act(name, z)[0], z, mag


def dense_residual_grad(dout, z, name="identity", gate=None, scale=1.0):
    """The elementwise part of the gradient: dz, dresidual, dbias, dgate (and the sums' magnitudes)."""
    M = dout.shape[0]
    a, d = act(name, z) if z is not None else (dout, np.ones_like(dout))
    g = gate_rows(gate, M)
    dz = dout * g * d
    r = {"dz": dz, "dresidual": scale * dout, "dbias": (dz.sum(0), np.abs(dz).sum(0))}
    if gate is not None:
        G = np.atleast_2d(gate).shape[0]
        r["dgate"] = _by_gate(dout * a, G), _by_gate(np.abs(dout * a), G)
    return r


def clip(grads, max_norm, eps):
    """(norm, factor)."""
    n = float(np.sqrt(sum(float((g * g).sum()) for g in grads)))
    return n, 1.0 if n + eps == 0 else min(1.0, max_norm / (n + eps))

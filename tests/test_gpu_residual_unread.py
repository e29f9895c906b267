"""Tensors that a call takes and does not read may be written by it: the same bits as with tensors apart."""

import pytest
import torch

import fp8_transformer_gb300 as te

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def n(g, *s, mean=0.0):
    return (torch.randn(*s, generator=g) + mean).to(BF).to(DEV)


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
def test_dy_in_the_place_of_y(norm):
    g = torch.Generator().manual_seed(1)
    M, H = 37, 264
    y, r, gamma, beta, dout, dxo = (n(g, M, H), n(g, M, H), n(g, H, mean=1.0), n(g, H), n(g, M, H), n(g, M, H))
    x, out = torch.empty_like(y), torch.empty_like(y)
    mu, rs = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    te.te_residual_norm_fwd(y, r, gamma, beta, x, out, norm_type=norm, mu=mu, rsigma=rs)
    got = []
    for dy in (torch.empty_like(y), y):
        dr, dg = torch.empty_like(y), torch.empty(H, device=DEV)
        te.te_residual_norm_bwd(dout, dxo, x, mu, rs, gamma, dr, dy, dg, y=y, norm_type=norm)
        got.append((dr, dy, dg))
    assert all(torch.equal(a, c) for a, c in zip(*got))


def test_dx_in_the_place_of_the_saved_z():
    g = torch.Generator().manual_seed(2)
    M, K = 40, 64
    x, w, dout, z = n(g, M, K), n(g, K, K), n(g, M, K), n(g, M, K)
    got = []
    for dx in (torch.empty_like(x), z):
        dw, db = torch.empty_like(w), torch.empty(K, device=DEV)
        te.te_dense_residual_bwd(dout, x, w, dx, dw, saved_z=z, dbias=db)
        got.append((dx, dw, db))
    assert all(torch.equal(a, c) for a, c in zip(*got))

"""te_dense_residual_bwd far from zero: values of z whose powers leave fp32, infinities and NaN.  One row, so that
dbias is dz itself in fp32 and dgate dout * act(z).

gelu'(z) and silu'(z) are 1 above 16 and 128, and 0 below -16 and -128, to 2^-24; act(z) is z or 0.  The
logistic of a far negative value is held at 2^-115 or less, not at 0, and what multiplies it in the derivative
is under 6000 (2 h sqrt(2 / pi) (1 + 3 * 0.044715 h^2) at 16): what stands for a zero is at most 6000 * 2^-115 of dout."""

import math

import pytest
import torch

import fp8_transformer_gb300 as te

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FAR = [130.0, 200.0, 1e5, 1e10, 1e11, 1e12, 1e13, 1e14, 1e19, 1e20, 1e30, 3e38, math.inf]


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_far_values(act):
    v = FAR + [-f for f in FAR] + [math.nan, 0.0]
    N, K = 32, 16
    z = torch.tensor([v + [0.5] * (N - len(v))], dtype=BF, device=DEV)
    dout = torch.linspace(-3, 3, N, device=DEV).to(BF)[None]
    x, w, gate = torch.ones(1, K, dtype=BF, device=DEV), torch.ones(K, N, dtype=BF, device=DEV), torch.ones(N, dtype=BF, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db, dg = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    te.te_dense_residual_bwd(dout, x, w, dx, dw, saved_z=z, activation=act, gate=gate, dbias=db, dgate=dg)
    d, n = dout[0].float(), len(FAR)
    zf = z[0].float()
    assert bool(((db[:n] - d[:n]).abs() <= 2.0 ** -22 * d[:n].abs()).all()), db[:n]
    finite = slice(0, n - 1)
    assert bool(((dg[finite] / zf[finite] - d[finite]).abs() <= 2.0 ** -22 * d[finite].abs()).all())
    assert bool(torch.isinf(dg[n - 1]))
    zero = 6000 * 2.0 ** -115 * 3
    assert bool((db[n:2 * n].abs() <= zero).all()) and bool((dg[n:2 * n].abs() <= zero).all())
    if act != "relu":  # relu of a NaN is 0 in this library
        assert bool(torch.isnan(db[2 * n])) and bool(torch.isnan(dg[2 * n]))
    assert torch.equal(dw[0], db.to(BF)) or torch.equal(torch.nan_to_num(dw[0]), torch.nan_to_num(db.to(BF)))

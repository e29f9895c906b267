"""How far te_grad_norm may be off, and its factor where the norm passes the largest fp32, on the GPU against exact
sums on the CPU.

A thread's squares of a chunk are added in fp32: of fp32 values each passes at most 7 roundings of 2^-24 (an end of
the tensor one, its chain 4, two where the chains meet), of bf16 values 11 (8 in the chain).  What comes after is
in pairs of fp32, whose errors (2^-48 of a sum) are 2^-20 of these at the lengths here.  The terms are
positive, so the sum is off by no more than that relative, the norm by half, and its rounding adds 2^-24."""

import math

import numpy as np
import pytest
import torch

import fp8_transformer_gb300 as te

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def exact(ts):
    """The norm, from a sum that is rounded once."""
    return math.sqrt(math.fsum(v * v for t in ts for v in t.cpu().double().tolist()))


@pytest.mark.parametrize("dtype,roundings", [(F32, 7), (BF, 11)])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 8, 31, 64, 333, 8192, 8200, 40001])
def test_norm_within_its_roundings(dtype, roundings, n):
    g = torch.Generator().manual_seed(n)
    norm = torch.empty(1, device=DEV)
    for offset in range(4):  # the ends that no vector covers
        for k in range(6):
            ts = [(torch.randn(n + offset, generator=g) * 10.0 ** (k - 3)).to(dtype).to(DEV)[offset:]]
            te.te_grad_norm(ts, norm)
            want = exact(ts)
            assert abs(norm.item() - want) <= (roundings / 2 + 1) * U * (1 + 2.0 ** -18) * want, (offset, k)


def test_a_norm_past_the_largest_fp32():
    """norm is an infinity then; the factor takes the norm as it was before it was rounded."""
    for dtype in (F32, BF):
        g = torch.tensor([3e38, -3e38, 1e30, 0.0], dtype=dtype, device=DEV)
        old = g.cpu().double().numpy()
        norm, out = torch.empty(1, device=DEV), torch.empty_like(g)
        te.te_grad_norm([g], norm)
        assert norm.item() == math.inf
        te.te_clip_grad_norm([g], 1e38, norm, outs=[out], epsilon=0.0)
        assert norm.item() == math.inf
        want = old * (1e38 / np.sqrt((old * old).sum()))
        # the factor's rounding, the norm's, the product's, and the type's: half a step each
        rel = 5.5 * U + 2 * U + torch.finfo(dtype).eps / 2
        assert (np.abs(out.cpu().double().numpy() - want) <= rel * np.abs(want)).all()
        te.te_clip_grad_norm([g], 1e39, norm, outs=[out])  # a limit above it: nothing changes
        assert torch.equal(out, g)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("std,max_norm", [(1e30, 1e-12), (1e36, 1e-8), (1e35, 3e-3), (1e37, 1e-20)])
def test_a_factor_below_the_normal_numbers(dtype, std, max_norm):
    """A factor of 2^-127 and less, which fp32 holds in few bits, on values that stay normal numbers."""
    g = torch.Generator().manual_seed(5)
    for offset in (0, 1):
        t = (torch.randn(5000, generator=g).clamp(-8, 8) * std).to(dtype).to(DEV)[offset:]
        norm, outs = torch.empty(1, device=DEV), [torch.empty(t.numel() + 8, dtype=dtype, device=DEV)]
        old = t.cpu().double().numpy()
        for at in (0, 3):  # places of the source's alignment and of another
            out = outs[0][at:at + t.numel()]
            te.te_clip_grad_norm([t], max_norm, norm, outs=[out], epsilon=0.0)
            want = old * (max_norm / np.sqrt((old * old).sum()))
            # as above; a value below the normal numbers may be off by two of its last places (2^-133 in bf16)
            last = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
            w = (7.5 * U + torch.finfo(dtype).eps / 2) * np.abs(want) + 2 * last
            assert (np.abs(out.cpu().double().numpy() - want) <= w).all()

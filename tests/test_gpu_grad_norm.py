"""te_grad_norm / te_clip_grad_norm on the GPU against float64.

A thread's squares of a chunk are added in fp32 (at most 11 roundings of 2^-24 on the way of any), the rest in
pairs that lose nothing of it, and the root halves that: the norm is within 2^-21 relative, its rounding
included, and the windows here are wider (2^-19).  A clipped value is one fp32 product with the rounded factor
(2^-20 from the norm, 2^-24 each) rounded to its type.
"""

import numpy as np
import pytest
import torch

import fp8_transformer_gb300 as te
from fp8_transformer_gb300 import dp
from oracle import numerics as nx
from oracle import residual as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
REL = 2.0 ** -19


def f64(t):
    return t.detach().cpu().double().numpy()


def grads(sizes, seed=0, std=0.01, dtypes=(BF, F32), offset=0):
    """Tensors cut from one buffer for each type, so that most start at odd places."""
    g = torch.Generator().manual_seed(seed)
    out = []
    bufs = {d: (torch.randn(sum(sizes) + len(sizes) + 8, generator=g) * std).to(d).to(DEV) for d in dtypes}
    at = {d: offset for d in dtypes}
    for i, n in enumerate(sizes):
        d = dtypes[i % len(dtypes)]
        out.append(bufs[d][at[d]:at[d] + n])
        at[d] += n
    return out


def check(gs, outs, norm, max_norm, eps=1e-6):
    old = [f64(t) for t in gs]
    n, c = orc.clip(old, max_norm, eps)
    assert abs(norm.item() - n) <= REL * n + 1e-45, (norm.item(), n)
    if outs is None:
        return
    for o, t in zip(old, outs):
        w = np.abs(o * c) * (REL + 2.0 ** -22)
        lo, hi = o * c - w, o * c + w
        if t.dtype == BF:
            lo, hi = nx.bf16_round(lo), nx.bf16_round(hi)
        got = f64(t)
        assert ((got >= lo) & (got <= hi)).all()


SIZES = [[1], [0], [8], [1, 0, 3, 0], [17, 4096, 5, 1, 8191, 8192, 8193], [100003], [1 << 20, 7],
         list(range(1, 40)), [129] * 700, [300000] * 3]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("max_norm", [0.05, 1e9, 0.0])
@pytest.mark.parametrize("offset", [0, 3])
def test_norm_and_clip(sizes, max_norm, offset):
    gs = grads(sizes, offset=offset)
    norm = torch.full((1,), 9.0, device=DEV)
    te.te_grad_norm(gs, norm)
    check(gs, None, norm, max_norm)
    outs = [torch.full((t.numel() + 9,), 5.0, dtype=t.dtype, device=DEV) for t in gs]
    views = [o[:t.numel()] for o, t in zip(outs, gs)]
    norm2 = torch.empty(1, device=DEV)
    te.te_clip_grad_norm(gs, max_norm, norm2, outs=views)
    assert torch.equal(norm, norm2)
    check(gs, views, norm2, max_norm)
    for o, t in zip(outs, gs):
        assert bool((o[t.numel():] == 5.0).all())
    # in place, through a list laid out beforehand: the same bits
    plan = te.GradList(gs)
    te.te_clip_grad_norm(plan, max_norm, norm2)
    assert torch.equal(norm, norm2)
    for o, t in zip(views, gs):
        assert torch.equal(o, t)


def test_neighbours_of_in_place_views_stay():
    buf = torch.randn(1000, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    old = buf.clone()
    te.te_clip_grad_norm([buf[13:500], buf[517:901]], 0.5, torch.empty(1, device=DEV))
    for a, b in ((0, 13), (500, 517), (901, 1000)):
        assert torch.equal(buf[a:b], old[a:b])
    assert not torch.equal(buf[13:500], old[13:500])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("std", [1e30, 1e18, 1e-18, 1e-24, 1e-36, 0.0])
def test_range(dtype, std):
    """Squares that overflow fp32, or vanish in it."""
    gs = grads([5000, 33], std=std, dtypes=(dtype,))
    gs.append(torch.zeros(4000, dtype=dtype, device=DEV))
    norm = torch.empty(1, device=DEV)
    te.te_grad_norm(gs, norm)
    check(gs, None, norm, 1.0)


def test_large_beside_small():
    gs = [torch.full((100000,), 1e-8, device=DEV), torch.tensor([1e20, 1.0], device=DEV), torch.full((999,), 1e-22, device=DEV)]
    norm = torch.empty(1, device=DEV)
    te.te_grad_norm(gs, norm)
    check(gs, None, norm, 1.0)
    te.te_grad_norm(gs[::2], norm)
    check(gs[::2], None, norm, 1.0)


@pytest.mark.parametrize("where", [0, 1, 5, 4097, 9999])
def test_nan_and_infinity(where):
    for bad in (float("nan"), float("inf"), float("-inf")):
        gs = grads([10000, 50], dtypes=(F32,))
        gs[0][where] = bad
        norm = torch.empty(1, device=DEV)
        te.te_clip_grad_norm(gs, 1.0, norm)
        if bad != bad:
            assert torch.isnan(norm).all() and all(bool(torch.isnan(t).all()) for t in gs)
        else:
            assert torch.isinf(norm).all() and bool(torch.isnan(gs[0][where]))
            assert bool((gs[1] == 0).all())


def test_zero_gradients_and_zero_epsilon():
    g = torch.zeros(300, device=DEV)
    norm = torch.empty(1, device=DEV)
    te.te_clip_grad_norm([g], 0.0, norm, epsilon=0.0)
    assert norm.item() == 0 and bool((g == 0).all())
    te.te_grad_norm([], norm.fill_(3.0))
    assert norm.item() == 0


def test_same_tensor_twice():
    g = torch.ones(100, device=DEV)
    norm = torch.empty(1, device=DEV)
    te.te_grad_norm([g, g], norm)  # reading: it counts twice
    assert abs(norm.item() - 200 ** 0.5) < 1e-5
    for a, o in (([g, g], None), ([g, g[50:]], None), ([g], [g[:100].view(100)]), ([g, g], [g, torch.empty_like(g)])):
        if o is not None and len(a) == 1:  # its own place is in place
            te.te_clip_grad_norm(a, 1e9, norm, outs=o)
            continue
        with pytest.raises(te.TEError):
            te.te_clip_grad_norm(a, 1.0, norm, outs=o)
    with pytest.raises(te.TEError):
        te.te_clip_grad_norm([g], 1.0, g[:1])


def test_a_list_whose_tensor_moved():
    p = torch.ones(50, device=DEV)
    plan = te.GradList([p])
    norm = torch.empty(1, device=DEV)
    te.te_grad_norm(plan, norm)
    p.data = torch.full((200,), 2.0, device=DEV)
    te.te_grad_norm(plan, norm)
    assert abs(norm.item() - 800 ** 0.5) < 1e-4
    p.data = torch.zeros(10)
    with pytest.raises(ValueError):
        te.te_grad_norm(plan, norm)


def test_streams_and_graphs():
    """Two captured calls replayed one after the other, with new values, each with its own workspace."""
    gs = grads([5000, 77, 300000])
    outs = [torch.empty_like(t) for t in gs]
    a, b = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    te.te_clip_grad_norm(gs, 0.1, a, outs=outs)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        te.te_clip_grad_norm(gs, 0.1, a, outs=outs)
    with torch.cuda.graph(g2):
        te.te_grad_norm(outs, b)
    for k in range(3):
        for t in gs:
            t.mul_(1.5)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        check(gs, outs, a, 0.1)
        check(outs, None, b, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = torch.empty(1, device=DEV)
    te.te_grad_norm(gs, c, stream=s)
    s.synchronize()
    te.te_grad_norm(gs, b)
    assert torch.equal(b, c)


def test_buckets():
    bk = dp.GradBuckets(64, 96, gated=True)
    g = torch.Generator().manual_seed(2)
    bk.weights.copy_(torch.randn(bk.weights.numel(), generator=g))
    bk.vectors.copy_(torch.randn(bk.vectors.numel(), generator=g))
    old = [bk.weights.clone(), bk.vectors.clone()]
    norm = bk.clip(2.0, torch.empty(1, device=DEV))
    check(old, [bk.weights, bk.vectors], norm, 2.0)


def test_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    g = torch.zeros((1 << 32) + 5, dtype=BF, device=DEV)
    g[-1], g[-70000], g[3] = 3.0, 4.0, 12.0
    norm = torch.empty(1, device=DEV)
    te.te_clip_grad_norm([g], 6.5, norm, epsilon=0.0)
    assert norm.item() == 13.0
    assert [g[i].item() for i in (-1, -70000, 3)] == [1.5, 2.0, 6.0]

"""te_residual_norm_fwd / _bwd on the GPU against the float64 oracle (oracle/residual.py).

Windows.  A row's sum passes at most 32 values in a thread, 5 steps of a warp and 32 warps: under 70
roundings of 2^-24, and a value is formed from two such statistics and some ten operations more, so an
fp32 value lies within W = 2^-17 of its terms' magnitudes.  What is stored is a rounding of a number in
that window (rounding is monotonic).  Column sums add one rounding for each of a CTA's rows (at most 10 in
these cases), 40 for the joined CTAs (32 terms and their own number / 32) and a few more:
W + 64 * 2^-24 < 2^-16 of the magnitudes.
"""

import ctypes

import numpy as np
import pytest
import torch

import fp8_transformer_gb300 as te
from oracle import numerics as nx
from oracle import residual as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
W, W_COL = 2.0 ** -17, 2.0 ** -16
BF, F32 = torch.bfloat16, torch.float32
GUARD = 64


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def within(name, got, ref, w, dtype=F32):
    lo, hi = ref - w, ref + w
    if dtype == BF:
        lo, hi = nx.bf16_round(lo), nx.bf16_round(hi)
    else:
        w32 = np.abs(ref) * 2.0 ** -24 + 2.0 ** -149
        lo, hi = lo - w32, hi + w32
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


def guarded(shape, dtype, keep):
    """A tensor with NaN (0xFF) bytes behind it; `keep` collects (whole, numel)."""
    n = int(np.prod(shape))
    whole = torch.full((n + GUARD,), float("nan") if dtype != torch.uint8 else 0xFF, dtype=dtype, device=DEV)
    keep.append((whole, n))
    return whole[:n].view(*shape)


def untouched(keep):
    for whole, n in keep:
        t = whole[n:]
        assert bool((t == 0xFF).all() if t.dtype == torch.uint8 else torch.isnan(t).all())


def draw(M, H, dt, rt, G, post, seed=0):
    g = torch.Generator().manual_seed(seed)

    def n(*s, std=1.0, mean=0.0, d=dt):
        return (torch.randn(*s, generator=g) * std + mean).to(d).to(DEV)

    t = dict(y=n(M, H, std=2.0), residual=n(M, H, std=3.0, mean=1.0, d=rt), gamma=n(H, std=0.3, mean=1.0),
             beta=n(H, std=0.3))
    if post:
        t.update(post_gamma=n(H, std=0.3, mean=1.0), post_beta=n(H, std=0.3))
    if G:
        t["gate"] = n(*((H,) if G == 1 else (G, H)), std=0.7)
    t["y"][0] *= 100.0
    if M > 2:
        t["residual"][2] += 300.0  # a mean far above the deviation
    return t, n


def run_fwd(t, ln, zc, out_dtype, scale, q=None, x_out=None, stream=None, residual=None):
    M, H = t["y"].shape
    keep = []
    r = residual if residual is not None else t["residual"]
    x = guarded((M, H), r.dtype, keep) if x_out is None else x_out
    out = guarded((M, H), out_dtype, keep)
    s = {k: guarded((M,), F32, keep) for k in ("mu", "rsigma")}
    if "post_gamma" in t:
        s.update({k: guarded((M,), F32, keep) for k in ("post_mu", "post_rsigma")})
    te.te_residual_norm_fwd(t["y"], r, t["gamma"], t["beta"] if ln else None, x, out,
                            norm_type="layernorm" if ln else "rmsnorm", zero_centered_gamma=zc, epsilon=1e-5,
                            post_gamma=t.get("post_gamma"), post_beta=t.get("post_beta") if ln else None,
                            gate=t.get("gate"), residual_scale=scale, q=q, stream=stream, **s)
    return x, out, s, keep


def oracle_fwd(t, ln, zc, scale):
    return orc.residual_norm_fwd(f64(t["y"]), f64(t["residual"]), f64(t["gamma"]), f64(t["beta"]),
                                 f64(t.get("post_gamma")), f64(t.get("post_beta")) if ln else None, f64(t.get("gate")),
                                 float(np.float32(scale)), ln, zc, float(np.float32(1e-5)))


def check_fwd(t, ln, zc, scale, x, out, s, want=None):
    want = want or oracle_fwd(t, ln, zc, scale)
    within("x_out", f64(x), *want["x_out"][:1], W * want["x_out"][1], x.dtype)
    if out.dtype != torch.uint8:
        within("out", f64(out), want["out"][0], W * want["out"][1], out.dtype)
    for m, r, src, wx in (("mu", "rsigma", want["x_out"][0], want["x_out"][1]),
                          ("post_mu", "post_rsigma", f64(t["y"]), None)):
        if m not in s or s[m] is None:
            continue
        a = np.abs(src).mean(1) if wx is None else wx.mean(1)
        within(m, f64(s[m]), want[m], W * a)
        d = np.abs(src - want[m][:, None])
        # rs moves by rs^3 mean(|d| e) with e the window of d
        e = (np.abs(src) if wx is None else wx) + np.abs(want[m][:, None])
        within(r, f64(s[r]), want[r], W * want[r] * (1 + want[r] ** 2 * (d * e).mean(1)))
    return want


SHAPES = [(1, 8), (1, 4096), (2, 64), (7, 1000), (33, 2048), (200, 136), (200, 1032), (200, 2056), (156, 8192), (1, 8192)]


@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("ln", [True, False])
@pytest.mark.parametrize("post", [True, False])
def test_forward(M, H, types, ln, post):
    G = 1 if M == 1 or M % 2 else (0 if post else 2)
    t, _ = draw(M, H, *types, G, post)
    x, out, s, keep = run_fwd(t, ln, post, types[0], 0.5 if post else 1.0)
    check_fwd(t, ln, post, 0.5 if post else 1.0, x, out, s)
    untouched(keep)


@pytest.mark.parametrize("M,H,ln,post", [(3, 4096, True, True), (200, 520, False, True), (160, 8192, True, False)])
@pytest.mark.parametrize("mode", ["delayed", "current"])
def test_forward_e4m3(M, H, ln, post, mode):
    t, _ = draw(M, H, BF, F32, 0, post)
    q = te.Quantizer(16.0, mode=mode)
    x, out, s, keep = run_fwd(t, ln, False, torch.uint8, 1.0, q)
    want = check_fwd(t, ln, False, 1.0, x, out, s)
    ref, w = want["out"][0], W * want["out"][1]
    amax = np.abs(ref).max()
    assert abs(q.amax.item() - amax) <= W * want["out"][1].max() + amax * 2.0 ** -23
    scale = q.scale.item()
    if mode == "current":
        assert scale == np.float32(448.0) / np.float32(q.amax.item())
    assert q.scale_inv.item() == np.float32(1.0) / np.float32(scale)
    w = w + np.abs(ref) * 2.0 ** -23
    lo, hi = (nx.e4m3_decode(nx.e4m3_encode((ref + d) * scale)) for d in (-w, w))
    got = nx.e4m3_decode(out.cpu().numpy())
    assert ((got >= lo) & (got <= hi)).all()
    untouched(keep)


def test_forward_amax_without_e4m3_and_fp32_out():
    t, _ = draw(5, 512, BF, BF, 0, False)
    q = te.Quantizer(1.0)
    x, out, s, _ = run_fwd(t, True, False, F32, 1.0, q)
    check_fwd(t, True, False, 1.0, x, out, s)
    assert q.amax.item() == out.abs().max().item()


@pytest.mark.parametrize("mode", [None, "current"])
@pytest.mark.parametrize("M", [3, 400])
def test_forward_in_place(M, mode):
    t, _ = draw(M, 1024, BF, BF, 1, True)
    q = te.Quantizer(1.0, mode=mode) if mode else None
    od = torch.uint8 if mode else BF
    x, out, _, _ = run_fwd(t, True, False, od, 1.0, q)
    r = t["residual"].clone()
    x2, out2, _, _ = run_fwd(t, True, False, od, 1.0, q, x_out=r, residual=r)
    assert torch.equal(x, r) and torch.equal(out, out2)


@pytest.mark.parametrize("G", [1, 4, 20])
def test_gates_take_their_rows(G):
    t, _ = draw(20, 256, BF, BF, 0, False)
    t["gate"] = torch.zeros(G, 256, dtype=BF, device=DEV)
    t["gate"] += torch.arange(1, G + 1, device=DEV, dtype=BF)[:, None]
    x, out, s, _ = run_fwd(t, True, False, BF, 1.0)
    check_fwd(t, True, False, 1.0, x, out, s)


def test_special_values():
    """A row's infinities and NaN stay in that row; a constant row has zero deviation."""
    t, _ = draw(6, 512, F32, F32, 0, True)
    t["y"][1, 7], t["residual"][3, 9] = float("inf"), float("nan")
    t["y"][4], t["residual"][4] = 2.0, 3.0
    for ln in (True, False):
        x, out, s, _ = run_fwd(t, ln, False, F32, 1.0)
        for r in (1, 3):
            assert bool(torch.isnan(out[r]).all())
        ok = [0, 2, 4, 5]
        sub = {k: (v[ok] if k in ("y", "residual") else v) for k, v in t.items()}
        check_fwd(sub, ln, False, 1.0, x[ok], out[ok], {k: v[ok] for k, v in s.items()})


# ------------------------------------------------------------------------------- backward ---


def run_bwd(t, n, ln, zc, scale, with_dxo=True, alias=False, stream=None, workspace=None):
    """Forward, backward, and the oracle's gradients from what the forward left."""
    M, H = t["y"].shape
    x, _, s, _ = run_fwd(t, ln, zc, t["y"].dtype, scale)
    dout, dxo = n(M, H), n(M, H, d=t["residual"].dtype) if with_dxo else None
    G = t["gate"].numel() // H if "gate" in t else 0
    post = "post_gamma" in t
    keep = []
    g = {k: guarded((H,), F32, keep) for k in ("dgamma", "dbeta") + (("dpost_gamma", "dpost_beta") if post else ())}
    if G:
        g["dgate"] = guarded(tuple(t["gate"].shape), F32, keep)
    dr = dxo.clone() if alias else guarded((M, H), t["residual"].dtype, keep)
    dy = guarded((M, H), t["y"].dtype, keep)
    te.te_residual_norm_bwd(dout, dr if alias else dxo, x, s["mu"] if ln else None, s["rsigma"], t["gamma"], dr, dy,
                            y=t["y"] if post or G else None, post_mu=s.get("post_mu") if ln else None,
                            post_rsigma=s.get("post_rsigma"), post_gamma=t.get("post_gamma"),
                            post_beta=t.get("post_beta") if ln else None, gate=t.get("gate"), residual_scale=scale,
                            norm_type="layernorm" if ln else "rmsnorm", zero_centered_gamma=zc, workspace=workspace,
                            stream=stream, **g)
    g.update(dresidual=dr, dy=dy)
    want = orc.residual_norm_bwd(f64(dout), f64(dxo), f64(x), f64(s["mu"]), f64(s["rsigma"]), f64(t["gamma"]),
                                 f64(t["y"]), f64(s.get("post_mu")), f64(s.get("post_rsigma")), f64(t.get("post_gamma")),
                                 f64(t.get("post_beta")) if ln else None, f64(t.get("gate")), float(np.float32(scale)),
                                 ln, zc)
    return g, want, keep


def check_bwd(g, want):
    for k, v in g.items():
        ref, mag = want[k]
        got = f64(v).reshape(ref.shape)
        within(k, got, ref, (W if k in ("dresidual", "dy") else W_COL) * mag, v.dtype)


@pytest.mark.parametrize("M,H", [(1, 8), (1, 4096), (6, 72), (33, 1000), (36, 2048), (400, 264), (156, 8192), (700, 1032)])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("ln", [True, False])
@pytest.mark.parametrize("post,G", [(True, 0), (True, 3), (False, 1), (False, 0)])
def test_backward(M, H, types, ln, post, G):
    G = G if M % max(G, 1) == 0 else 1
    t, n = draw(M, H, *types, G, post)
    g, want, keep = run_bwd(t, n, ln, post, 0.5 if G else 1.0, with_dxo=G != 1)
    check_bwd(g, want)
    untouched(keep)


@pytest.mark.parametrize("M,G", [(768, 4), (600, 600), (640, 40), (96, 48), (1000, 2)])
def test_backward_gates(M, G):
    """Gates whose rows several CTAs share, and CTAs that hold several gates' rows."""
    t, n = draw(M, 1032, BF, BF, G, True)
    g, want, keep = run_bwd(t, n, True, False, 1.0)
    check_bwd(g, want)
    untouched(keep)


def test_backward_in_place_and_again():
    t, n = draw(300, 512, BF, BF, 1, True)
    a, _, _ = run_bwd(t, n, True, False, 1.0)
    t, n = draw(300, 512, BF, BF, 1, True)
    b, _, _ = run_bwd(t, n, True, False, 1.0, alias=True)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_no_rows_zero_the_sums():
    H, z = 64, lambda *s, d=BF: torch.empty(*s, dtype=d, device=DEV)  # noqa: E731
    v = {k: torch.full((H,), 7.0, device=DEV) for k in ("dgamma", "dbeta", "dpost_gamma", "dpost_beta")}
    dg = torch.full((3, H), 7.0, device=DEV)
    te.te_residual_norm_bwd(z(0, H), None, z(0, H), z(0, d=F32), z(0, d=F32), z(H), None, z(0, H), y=z(0, H),
                            post_mu=z(0, d=F32), post_rsigma=z(0, d=F32), post_gamma=z(H), gate=z(3, H), dgate=dg, **v)
    assert all(bool((t == 0).all()) for t in (dg, *v.values()))
    te.te_residual_norm_fwd(z(0, H), z(0, H), z(H), None, z(0, H), z(0, H), gate=z(3, H))


def test_gradient_against_differences():
    """The whole chain in fp32: the directional derivative of a scalar of the forward pass."""
    M, H = 12, 256
    t, n = draw(M, H, F32, F32, 3, True, seed=4)
    t["y"][0] /= 100.0
    t["residual"][2] -= 300.0
    g, _, _ = run_bwd(t, n, True, False, 0.5)
    t2, n2 = draw(M, H, F32, F32, 3, True, seed=4)  # the same draw again gives the same upstream gradients
    dout, dxo = f64(n2(M, H)), f64(n2(M, H))
    leaves = dict(y="dy", residual="dresidual", gamma="dgamma", beta="dbeta", post_gamma="dpost_gamma",
                  post_beta="dpost_beta", gate="dgate")
    a = {k: f64(t[k]) for k in leaves}

    def value(v):
        f = orc.residual_norm_fwd(v["y"], v["residual"], v["gamma"], v["beta"], v["post_gamma"], v["post_beta"],
                                  v["gate"], 0.5, True, False, float(np.float32(1e-5)))
        return float((f["out"][0] * dout).sum() + (f["x_out"][0] * dxo).sum())

    r = np.random.default_rng(0)
    for leaf, grad in leaves.items():
        d = r.normal(size=a[leaf].shape)
        h = 1e-5
        diff = (value({**a, leaf: a[leaf] + h * d}) - value({**a, leaf: a[leaf] - h * d})) / (2 * h)
        got = float((f64(g[grad]) * d).sum())
        # the GPU's gradient is within W_COL of its terms; the differences' own error is far below
        assert abs(got - diff) <= 1e-4 * float(np.abs(f64(g[grad]) * d).sum()) + 1e-6, leaf


def test_streams_graphs_and_host_threads():
    """On another stream, captured with other inputs at replay, and with a workspace of the caller's."""
    t, n = draw(64, 1024, BF, BF, 2, True)
    base, _, _ = run_bwd(t, n, True, False, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t, n = draw(64, 1024, BF, BF, 2, True)
    with torch.cuda.stream(s):
        other, _, _ = run_bwd(t, n, True, False, 1.0)
    s.synchronize()
    for k in base:
        assert torch.equal(base[k], other[k]), k
    x, out = torch.empty_like(t["y"]), torch.empty_like(t["y"])
    args = (t["y"], t["residual"], t["gamma"], t["beta"], x, out)
    kw = dict(post_gamma=t["post_gamma"], post_beta=t["post_beta"], gate=t["gate"])
    te.te_residual_norm_fwd(*args, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        te.te_residual_norm_fwd(*args, **kw)
    t["y"].mul_(-0.5)
    want_x, want_out = torch.empty_like(x), torch.empty_like(out)
    te.te_residual_norm_fwd(t["y"], t["residual"], t["gamma"], t["beta"], want_x, want_out, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want_x) and torch.equal(out, want_out)


def test_amax_in_a_graph():
    """The amax is zeroed by every replay, beside the kernel that takes it."""
    t, n = draw(37, 1024, BF, BF, 0, True)
    x, out = torch.empty_like(t["y"]), torch.empty(37, 1024, dtype=torch.uint8, device=DEV)
    q = te.Quantizer(16.0)
    args = (t["y"], t["residual"], t["gamma"], t["beta"], x, out)
    kw = dict(post_gamma=t["post_gamma"], post_beta=t["post_beta"], q=q)
    te.te_residual_norm_fwd(*args, **kw)
    first = q.amax.item()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        te.te_residual_norm_fwd(*args, **kw)
        copy = q.amax.clone()
    q.amax.fill_(1e9)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert copy.item() == first == q.amax.item()
    t["gamma"].mul_(0.5)
    t["beta"].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert copy.item() == pytest.approx(first / 2, rel=2.0 ** -20)


def test_two_host_threads():
    """Calls of two threads on streams of their own, each with its own kept workspace."""
    import threading
    t, n = draw(48, 512, BF, BF, 2, True)
    want, _, _ = run_bwd(t, n, True, False, 1.0)
    got, errors = {}, []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    tt, nn = draw(48, 512, BF, BF, 2, True)
                    torch.cuda.current_stream().synchronize()
                    got[k], _, _ = run_bwd(tt, nn, True, False, 1.0)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [h.start() for h in threads]
    [h.join() for h in threads]
    assert not errors
    for k in range(2):
        for name in want:
            assert torch.equal(want[name], got[k][name]), name


@pytest.mark.parametrize("H", [64, 1024, 4096])
def test_many_rows_to_a_cta(H):
    """Rows far beyond the ring, their number no multiple of anything, gates that end anywhere."""
    M = 9009 if H < 4096 else 3003
    t, n = draw(M, H, BF, BF, 3, True)
    x, out, s, _ = run_fwd(t, True, False, BF, 1.0)
    check_fwd(t, True, False, 1.0, x, out, s)
    g, want, _ = run_bwd(t, n, True, False, 1.0)
    check_bwd(g, want)


def test_workspace_is_checked():
    t, n = draw(40, 256, BF, BF, 0, False)
    need = te.lib().te_residual_norm_bwd_workspace(40, 256, 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    g, want, _ = run_bwd(t, n, True, False, 1.0, workspace=ws)
    check_bwd(g, want)
    with pytest.raises(te.TEError):
        run_bwd(t, n, True, False, 1.0, workspace=ws[:need - 16])
    assert ctypes.c_size_t(need).value > 0


def test_offsets_past_32_bits():
    """More than 2^32 bytes (and 2^31 elements) in a tensor: the last rows, forward and backward."""
    H = 8192
    M = (1 << 31) // H + 8
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    y = torch.zeros(M, H, dtype=BF, device=DEV)
    r = torch.zeros(M, H, dtype=BF, device=DEV)
    t, n = draw(8, H, BF, BF, 0, False)
    y[-8:], r[-8:] = t["y"], t["residual"]
    x, out = torch.empty_like(y), torch.empty_like(y)
    mu, rsig = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    te.te_residual_norm_fwd(y, r, t["gamma"], t["beta"], x, out, mu=mu, rsigma=rsig, epsilon=1e-5)
    check_fwd(t, True, False, 1.0, x[-8:], out[-8:], dict(mu=mu[-8:], rsigma=rsig[-8:]))
    dout, dy = torch.zeros_like(y), out  # the forward's result is not needed again
    dout[-8:] = n(8, H)
    dg, db = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    te.te_residual_norm_bwd(dout, None, x, mu, rsig, t["gamma"], None, dy, dg, db)
    want = orc.residual_norm_bwd(f64(dout[-8:]), None, f64(x[-8:]), f64(mu[-8:]), f64(rsig[-8:]), f64(t["gamma"]))
    within("dy", f64(dy[-8:]), want["dy"][0], W * want["dy"][1], BF)
    within("dgamma", f64(dg), want["dgamma"][0], W_COL * want["dgamma"][1])
    within("dbeta", f64(db), want["dbeta"][0], W_COL * want["dbeta"][1])

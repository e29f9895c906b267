"""te_dense_residual_fwd / _bwd on the GPU against the float64 oracle (oracle/residual.py).

Windows, as for the other products (an accumulation is within 2^-18 of the sum of the products'
magnitudes; activations and their derivatives within 1e-5 of the terms that form them): z = product +
bias within WZ = 2^-18 |x| |w| + 2^-22 (|z| + |b|), act(z) within 1.2 WZ + 1e-5 |z| (no activation here
is steeper than 1.13), and what joins the stream adds 2^-22 of its terms.  What is stored is a rounding
of a number in the window.  dz is rounded before the products: where its window holds a border, the
product may see the value on either side, and the jump counts through the operand's magnitudes.  Column
sums pass at most 32 rows in a warp, 8 warps, chunks and 16 warps again: 2^-17 of their terms.
"""

import numpy as np
import pytest
import torch

import fp8_transformer_gb300 as te
from oracle import numerics as nx
from oracle import residual as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
ACC, ACT, COL = 2.0 ** -18, 1e-5, 2.0 ** -17


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def within(name, got, ref, w, dtype):
    lo, hi = ref - w, ref + w
    if dtype == BF:
        lo, hi = nx.bf16_round(lo), nx.bf16_round(hi)
    else:
        d = np.abs(ref) * 2.0 ** -23 + 2.0 ** -140
        lo, hi = lo - d, hi + d
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


def draw(M, K, N, fp8=False, G=0, bias=True, rt=BF, seed=0):
    g = torch.Generator().manual_seed(seed)

    def n(*s, std=1.0, mean=0.0, d=BF):
        return (torch.randn(*s, generator=g) * std + mean).to(d).to(DEV)

    t = dict(x=n(M, K), w=n(K, N, std=0.05), residual=n(M, N, std=3.0, d=rt), bias=n(N) if bias else None,
             gate=n(*((N,) if G == 1 else (G, N)), std=0.7) if G else None, x_inv=None, w_inv=None)
    if fp8:
        for k, s in (("x", 64.0), ("w", 1024.0)):
            t[k] = (t[k].float() * s).clamp(-448, 448).to(torch.float8_e4m3fn)
            t[k + "_inv"] = torch.tensor([1 / s], device=DEV)
    return t, n


def values(t):
    """x and w as float64, with their factors."""
    x, w = f64(t["x"].float()), f64(t["w"].float())
    if t["x_inv"] is not None:
        x, w = x * t["x_inv"].item(), w * t["w_inv"].item()
    return x, w


def run_fwd(t, act, scale, save=True, out=None, residual=None, **kw):
    r = t["residual"] if residual is None else residual
    M, N = r.shape
    whole = torch.full((M * N + 64,), float("nan"), dtype=r.dtype, device=DEV)
    out = whole[:M * N].view(M, N) if out is None else out
    z = torch.empty(M, N, dtype=BF, device=DEV) if save else None
    te.te_dense_residual_fwd(t["x"], t["w"], r, out, bias=t["bias"], activation=act, gate=t["gate"],
                             residual_scale=scale, saved_z=z, x_scale_inv=t["x_inv"], kernel_scale_inv=t["w_inv"], **kw)
    assert bool(torch.isnan(whole[M * N:]).all())
    return out, z


def check_fwd(t, act, scale, out, z, rows=None):
    x, w = values(t)
    res, gate = f64(t["residual"]), f64(t["gate"])
    M = x.shape[0]
    ref, rz, mag = orc.dense_residual_fwd(x, w, res, f64(t["bias"]), act, gate, scale)
    b = 0.0 if t["bias"] is None else np.abs(f64(t["bias"]))
    wz = ACC * mag + 2.0 ** -22 * (np.abs(rz) + b)
    g = np.abs(orc.gate_rows(gate, M))
    wa = wz if act == "identity" else 1.2 * wz + ACT * np.abs(rz)
    a = np.abs(orc.act(act, rz)[0])
    within("out", f64(out), ref, g * wa + 2.0 ** -22 * (np.abs(scale * res) + g * a), out.dtype)
    if z is not None:
        within("z", f64(z), rz, wz, BF)


SHAPES = [(1, 16, 16), (1, 4096, 4096), (2, 512, 48), (5, 1040, 272), (8, 2064, 4096), (9, 64, 1008), (16, 4096, 512),
          (17, 1024, 640), (31, 96, 8192), (33, 14336, 256), (64, 256, 64), (65, 528, 272), (129, 512, 528), (130, 1024, 1024),
          (257, 80, 16), (300, 4096, 784), (16, 64, 28672), (9, 4096, 32), (24, 160, 14336), (32, 8192, 80)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rt", [BF, F32])
def test_forward(M, K, N, fp8, rt):
    i = SHAPES.index((M, K, N))
    act = ["identity", "gelu", "silu", "relu"][i % 4]
    G = [0, 1, M][i % 3] if M < 100 else [0, 1][i % 2]
    t, _ = draw(M, K, N, fp8, G, bias=i % 2 == 0, rt=rt)
    scale = 0.5 if i % 3 else 1.0
    out, z = run_fwd(t, act, scale, save=i % 4 != 0)
    check_fwd(t, act, scale, out, z)


@pytest.mark.parametrize("act", ["identity", "relu", "gelu", "silu"])
@pytest.mark.parametrize("G", [0, 1, 4])
@pytest.mark.parametrize("M", [8, 192])
def test_forward_every_epilogue(act, G, M):
    t, _ = draw(M, 512, 528, False, G)
    out, z = run_fwd(t, act, 0.25)
    check_fwd(t, act, 0.25, out, z)


@pytest.mark.parametrize("M", [1, 3, 40, 200])
def test_forward_in_place_and_again(M):
    t, _ = draw(M, 1024, 512, False, 1)
    out, _ = run_fwd(t, "gelu", 1.0)
    r = t["residual"].clone()
    got, _ = run_fwd(t, "gelu", 1.0, out=r, residual=r)
    assert torch.equal(out, got)


@pytest.mark.parametrize("M", [1, 6, 20, 140])
def test_rows_do_not_touch_one_another(M):
    """An infinity or a NaN of one row of x stays in that row; of the residual, in its place."""
    t, _ = draw(M, 256, 160)
    out, _ = run_fwd(t, "identity", 1.0)
    t["x"][M - 1, 3] = float("nan")
    t["residual"][0, 5] = float("inf")
    got, _ = run_fwd(t, "identity", 1.0)
    assert bool(torch.isnan(got[M - 1]).all())
    if M > 1:
        assert bool(torch.isinf(got[0, 5]))
        out[0, 5] = got[0, 5]
        assert torch.equal(out[:M - 1], got[:M - 1])


# outputs of many tiles, which the batch product's kernel makes whatever K is
MANY = [(257, 80, 16384), (2500, 96, 1040), (70, 64, 28672), (5000, 16, 528), (1300, 1040, 2064), (4099, 128, 592)]


@pytest.mark.parametrize("M,K,N", MANY)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rt", [BF, F32])
def test_forward_many_tiles(M, K, N, fp8, rt):
    i = MANY.index((M, K, N))
    act = ["gelu", "identity", "relu", "silu"][i % 4]
    t, _ = draw(M, K, N, fp8, [1, 4, 0, 8, 13, 0][i], bias=i % 2 == 0, rt=rt)
    out, z = run_fwd(t, act, 0.5, save=i % 3 != 2)
    check_fwd(t, act, 0.5, out, z)
    r = t["residual"].clone()
    again, _ = run_fwd(t, act, 0.5, out=r, residual=r)
    assert torch.equal(out, again)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        t["x"][M - 1] = float("nan")
        other, _ = run_fwd(t, act, 0.5)
    s.synchronize()
    assert torch.equal(out[:M - 1], other[:M - 1]) and (act == "relu" or bool(torch.isnan(other[M - 1]).all()))


# outputs of few tiles: every width of a tile, ends of K inside a stage, clusters of one to eight
FEW = [(32, 16, 16), (32, 16400, 144), (33, 80, 1040), (48, 1168, 272), (64, 4112, 128), (63, 128, 19456), (65, 16, 4096),
       (96, 2064, 2064), (128, 14336, 144), (127, 256, 9600), (129, 640, 400), (255, 4112, 272), (700, 208, 160),
       (1025, 1024, 1024), (2000, 48, 16)]


@pytest.mark.parametrize("M,K,N", FEW)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rt", [BF, F32])
def test_forward_few_tiles(M, K, N, fp8, rt):
    i = FEW.index((M, K, N))
    act = ["silu", "gelu", "identity", "relu"][i % 4]
    t, _ = draw(M, K, N, fp8, [0, 1, M][i % 3], bias=i % 2 == 0, rt=rt)
    out, z = run_fwd(t, act, 0.5, save=i % 3 != 2)
    check_fwd(t, act, 0.5, out, z)
    for _ in range(3):  # the same sums in the same order every time
        r = t["residual"].clone()
        again, _ = run_fwd(t, act, 0.5, out=r, residual=r)
        assert torch.equal(out, again)


@pytest.mark.parametrize("M", [20, 50, 120, 300])
def test_layers_one_after_another(M):
    """Each layer may start while the one in front ends: a chain of few tiles, of many tiles, and a norm between
    them gives what the layers give one by one."""
    t, n = draw(M, 1024, 1024, False, 1)
    wide, back = n(1024, 28672, std=0.03), n(28672, 1024, std=0.01)
    r_wide = n(M, 28672)
    gamma, beta = n(1024, std=0.1, mean=1.0), n(1024, std=0.1)

    def chain(wait):
        x = t["x"]
        for _ in range(4):
            for w, r in ((t["w"], t["residual"]), (wide, r_wide), (back, t["residual"])):
                out = torch.empty_like(r)
                te.te_dense_residual_fwd(x, w, r, out, activation="silu", residual_scale=0.5)
                wait()
                x = out
            out, ln = torch.empty_like(x), torch.empty_like(x)
            te.te_residual_norm_fwd(x, t["residual"], gamma, beta, out, ln)
            wait()
            x = ln
        return x

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(chain(lambda: None), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(lambda: None)
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


# ------------------------------------------------------------------------------- backward ---


def bwd(t, n, act, scale, z, rt=BF, q=None, want_dr=True, workspace=None, stream=None):
    M, K = t["x"].shape
    N = t["w"].shape[1]
    g = t.get("dout")
    dout = n(M, N, d=rt) if g is None else g
    o = dict(dx=torch.empty(M, K, dtype=BF, device=DEV), dkernel=torch.empty(K, N, dtype=BF, device=DEV),
             dbias=torch.empty(N, device=DEV), dresidual=torch.empty(M, N, dtype=rt, device=DEV) if want_dr else None,
             dgate=torch.empty(t["gate"].shape, device=DEV) if t["gate"] is not None else None)
    te.te_dense_residual_bwd(dout, t["x"], t["w"], o["dx"], o["dkernel"], dresidual=o["dresidual"], saved_z=z,
                             activation=act, gate=t["gate"], residual_scale=scale, dbias=o["dbias"], dgate=o["dgate"],
                             q=q, x_scale_inv=t["x_inv"], kernel_scale_inv=t["w_inv"], workspace=workspace, stream=stream)
    return dout, o


def check_bwd(t, act, scale, z, dout, o, q=None):
    x, w = values(t)
    d, zz, gate = f64(dout), f64(z), f64(t["gate"])
    M = x.shape[0]
    r = orc.dense_residual_grad(d, zz, act, gate, scale)
    g = np.abs(orc.gate_rows(gate, M))
    dz = r["dz"]
    wd = np.abs(dz) * 2.0 ** -22 + (0.0 if act == "identity" else np.abs(d) * g * ACT * (1 + np.abs(zz)))
    if q is None:
        lo, mid, hi = (nx.bf16_round(v) for v in (dz - wd, dz, dz + wd))
    else:
        s, inv = q.scale.item(), q.scale_inv.item()
        lo, mid, hi = (nx.e4m3_decode(nx.e4m3_encode(v * s)) * inv for v in (dz - wd, dz, dz + wd))
    jump = np.maximum(hi - mid, mid - lo)
    for name, ref, mag, j in (("dx", mid @ w.T, np.abs(mid) @ np.abs(w.T), jump @ np.abs(w.T)),
                              ("dkernel", x.T @ mid, np.abs(x.T) @ np.abs(mid), np.abs(x.T) @ jump)):
        within(name, f64(o[name]), ref, ACC * mag + 2.0 ** -22 * np.abs(ref) + j, BF)
    within("dbias", f64(o["dbias"]), r["dbias"][0], COL * r["dbias"][1] + wd.sum(0), F32)
    if o["dgate"] is not None:
        G = np.atleast_2d(gate).shape[0]
        wa = 0.0 if act == "identity" else (np.abs(d) * ACT * np.abs(zz)).reshape(G, -1, d.shape[1]).sum(1)
        within("dgate", f64(o["dgate"]).reshape(G, -1), r["dgate"][0], COL * r["dgate"][1] + wa, F32)
    if o["dresidual"] is not None:
        within("dresidual", f64(o["dresidual"]), r["dresidual"], 0.0, o["dresidual"].dtype)


@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (7, 512, 272), (128, 64, 528), (260, 272, 1040), (516, 512, 256)])
@pytest.mark.parametrize("act", ["identity", "relu", "gelu", "silu"])
@pytest.mark.parametrize("G", [0, 1, 4])
@pytest.mark.parametrize("rt", [BF, F32])
def test_backward(M, K, N, act, G, rt):
    G = G if M % max(G, 1) == 0 else 1
    t, n = draw(M, K, N, False, G, rt=rt)
    z = n(M, N, std=2.0) if act != "identity" or G else None
    dout, o = bwd(t, n, act, 0.5, z, rt, want_dr=G != 1)
    check_bwd(t, act, 0.5, z, dout, o)


@pytest.mark.parametrize("M,G", [(5, 5), (1000, 500), (1300, 1300), (390, 3)])
def test_backward_gates(M, G):
    """More gates than the summing kernel has CTAs, and gates of odd numbers of rows."""
    t, n = draw(M, 32, 272, False, G)
    z = n(M, 272, std=2.0)
    dout, o = bwd(t, n, "silu", 1.0, z)
    check_bwd(t, "silu", 1.0, z, dout, o)


@pytest.mark.parametrize("mode", ["delayed", "current"])
@pytest.mark.parametrize("act,G,M", [("gelu", 2, 130), ("identity", 0, 33), ("relu", 1, 260)])
def test_backward_fp8(mode, act, G, M):
    t, n = draw(M, 256, 528, True, G)
    z = n(M, 528, std=2.0) if act != "identity" or G else None
    q = te.Quantizer(40.0, mode=mode)
    dout, o = bwd(t, n, act, 1.0, z, q=q)
    r = orc.dense_residual_grad(f64(dout), f64(z), act, f64(t["gate"]), 1.0)
    amax = np.abs(r["dz"]).max()
    assert abs(q.amax.item() - amax) <= 3e-5 * amax
    if mode == "current":
        assert q.scale.item() == np.float32(448.0) / np.float32(q.amax.item())
    assert q.scale_inv.item() == np.float32(1.0) / np.float32(q.scale.item())
    check_bwd(t, act, 1.0, z, dout, o, q)


def test_forward_and_backward_together():
    """A step of the layer as it is used: the forward's saved z and stream, the gradients of all that it
    read, held to differences of the oracle's forward along a random direction."""
    M, K, N, G = 24, 64, 96, 3
    t, n = draw(M, K, N, False, G, rt=F32)
    out, z = run_fwd(t, "gelu", 0.5)
    dout, o = bwd(t, n, "gelu", 0.5, z, F32)
    check_bwd(t, "gelu", 0.5, z, dout, o)
    x, w = values(t)
    leaves = {"x": (x, "dx"), "w": (w, "dkernel"), "residual": (f64(t["residual"]), "dresidual"),
              "bias": (f64(t["bias"]), "dbias"), "gate": (f64(t["gate"]), "dgate")}

    def value(v):
        return float((orc.dense_residual_fwd(v["x"], v["w"], v["residual"], v["bias"], "gelu", v["gate"], 0.5)[0]
                      * f64(dout)).sum())

    r = np.random.default_rng(1)
    base = {k: v[0] for k, v in leaves.items()}
    for k, (v, grad) in leaves.items():
        d = r.normal(size=v.shape)
        diff = (value({**base, k: v + 1e-6 * d}) - value({**base, k: v - 1e-6 * d})) / 2e-6
        got = f64(o[grad]) * d
        # z is stored in bf16: half a step of it moves act' by at most 2^-9 |z|, |act''| < 1.2 and |z| < 5 here;
        # dz and the products' outputs are rounded by 2^-8 of themselves at most
        assert abs(got.sum() - diff) <= (6 * 2.0 ** -8 + 2 * 2.0 ** -8) * np.abs(got).sum(), k


def test_no_rows():
    z = lambda *s, d=BF: torch.empty(*s, dtype=d, device=DEV)  # noqa: E731
    te.te_dense_residual_fwd(z(0, 64), z(64, 32), z(0, 32), z(0, 32))
    dk, db, dg = z(64, 32).fill_(3), z(32, d=F32).fill_(3), z(2, 32, d=F32).fill_(3)
    te.te_dense_residual_bwd(z(0, 32), z(0, 64), z(64, 32), z(0, 64), dk, gate=z(2, 32), saved_z=z(0, 32), dbias=db, dgate=dg)
    assert all(bool((v == 0).all()) for v in (dk, db, dg))


# (the last five: the first product on many tiles, the same split along K, on single rows of tiles; the second product
# split; and neither)
BESIDE = [(1, 64, 64), (48, 2064, 4112), (128, 528, 2064), (20, 9616, 80), (130, 1024, 1024), (2100, 2048, 1040),
          (2100, 2048, 80), (2304, 1024, 8192), (100, 20480, 64), (17000, 64, 256), (700, 8192, 272)]


@pytest.mark.parametrize("M,K,N", BESIDE)
@pytest.mark.parametrize("fp8", [False, True])
def test_backward_products_beside_one_another(M, K, N, fp8):
    """The second product of a call starts while the first ends, and the next call reuses the workspace: calls on
    two sets of inputs in turn, without a wait, give what each gives by itself, eager and from a graph."""
    sets = []
    for k in range(2):
        t, n = draw(M, K, N, fp8, 1, seed=k)
        t["dout"] = n(M, N)
        _, z = run_fwd(t, "gelu", 1.0)
        sets.append((t, n, z, te.Quantizer(40.0, mode="current") if fp8 else None))

    def call(k):
        t, n, z, q = sets[k]
        return bwd(t, n, "gelu", 1.0, z, q=q)[1]

    want = []
    for k in range(2):
        want.append(call(k))
        torch.cuda.synchronize()
    t, _, z, q = sets[1]
    check_bwd(t, "gelu", 1.0, z, t["dout"], want[1], q)
    got = [call(i % 2) for i in range(8)]
    # what follows on the stream sees both products' results
    sums = [o["dx"].double().sum() + o["dkernel"].double().sum() for o in got]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(o[name], want[i % 2][name]) for name in o if o[name] is not None)
        assert sums[i] == want[i % 2]["dx"].double().sum() + want[i % 2]["dkernel"].double().sum()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [call(i % 2) for i in range(4)]
    for _ in range(3):
        for o in out:
            o["dx"].zero_(), o["dkernel"].zero_()
        g.replay()
    torch.cuda.synchronize()
    for i, o in enumerate(out):
        assert all(torch.equal(o[name], want[i % 2][name]) for name in o if o[name] is not None)


@pytest.mark.parametrize("M", [1, 12, 200])
def test_streams_and_graphs(M):
    t, n = draw(M, 2048, 512, False, 1)
    out, z = run_fwd(t, "silu", 1.0)
    dout, o = bwd(t, n, "silu", 1.0, z)
    t["dout"] = dout
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out2, z2 = run_fwd(t, "silu", 1.0)
        _, o2 = bwd(t, n, "silu", 1.0, z2)
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(z, z2)
    assert all(torch.equal(o[k], o2[k]) for k in o)
    # two graphs of one shape, replayed in turn on new inputs
    outs, graphs = [torch.empty_like(out) for _ in range(2)], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            te.te_dense_residual_fwd(t["x"], t["w"], t["residual"], outs[k], bias=t["bias"], activation="silu",
                                     gate=t["gate"])
        graphs.append(g)
    t["x"].mul_(0.5)
    want, _ = run_fwd(t, "silu", 1.0)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_backward_of_very_many_columns():
    """More than 65535 strips of 256 columns; whole numbers, whose sums are exact in any order."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    M, K, N = 2, 16, 65537 * 256 + 16
    g = torch.Generator(device=DEV).manual_seed(3)

    def few(*s, d=BF):
        return torch.randint(-1, 2, s, generator=g, device=DEV, dtype=torch.int8).to(d)

    x, w, dout, z, gate = few(M, K), few(K, N), few(M, N), few(M, N), few(N)
    dx, dw, dres = torch.empty_like(x), torch.empty_like(w), torch.empty_like(dout)
    db, dg = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    te.te_dense_residual_bwd(dout, x, w, dx, dw, dresidual=dres, saved_z=z, activation="relu", gate=gate, residual_scale=0.5,
                             dbias=db, dgate=dg)
    dz = (dout * gate * (z > 0)).float()
    assert torch.equal(db, dz.sum(0)) and torch.equal(dg, (dout * z.clamp(min=0)).float().sum(0))
    assert torch.equal(dres, dout * 0.5)
    assert torch.equal(dw, (x[0, :, None] * dz[0] + x[1, :, None] * dz[1]).to(BF))
    want = torch.stack([(w[k].float() * dz).double().sum(1) for k in range(K)], 1)
    assert torch.equal(dx, want.float().to(BF))


def test_workspaces():
    """A workspace that stops short of the scratch for splitting serves; a shorter one is refused."""
    t, n = draw(200, 4096, 256)
    z = None
    dout, o = bwd(t, n, "identity", 1.0, z)
    t["dout"] = dout
    need = te.lib().te_dense_residual_bwd_workspace(200, 4096, 256, 1, te.binding.TE_BF16)
    gemm = te.binding.TE_OP_GEMM  # the scratch that each of the two products would use: {M, K, N}
    split = max(te.workspace_size(gemm, 200, 256, 4096), te.workspace_size(gemm, 4096, 200, 256))
    for size in (need, need - (split + 255) // 256 * 256):
        _, o2 = bwd(t, n, "identity", 1.0, z, workspace=torch.empty(size, dtype=torch.uint8, device=DEV))
        check_bwd(t, "identity", 1.0, z, dout, o2)
    with pytest.raises(te.TEError):
        bwd(t, n, "identity", 1.0, z, workspace=torch.empty(4096, dtype=torch.uint8, device=DEV))


def test_a_layer_step_end_to_end():
    """The set as a training step uses it: residual norm, the dense layer into the stream, both gradients and
    the clipping of what they leave, against the same chain of the oracle from the tensors that each stored."""
    M, H = 96, 256
    t, n = draw(M, H, H, False, 1)
    y, gamma, beta = n(M, H), n(H, std=0.1, mean=1.0), n(H, std=0.1)
    x1, ln = torch.empty(M, H, dtype=BF, device=DEV), torch.empty(M, H, dtype=BF, device=DEV)
    mu, rs = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    te.te_residual_norm_fwd(y, t["residual"], gamma, beta, x1, ln, mu=mu, rsigma=rs)
    out, z = torch.empty_like(x1), torch.empty_like(x1)
    te.te_dense_residual_fwd(ln, t["w"], x1, out, bias=t["bias"], activation="gelu", gate=t["gate"], saved_z=z)
    check_fwd({**t, "x": ln, "residual": x1}, "gelu", 1.0, out, z)
    dout = n(M, H)
    dln, dw = torch.empty_like(ln), torch.empty_like(t["w"])
    db, dgate, dg, dbeta = (torch.empty(H, device=DEV) for _ in range(4))
    te.te_dense_residual_bwd(dout, ln, t["w"], dln, dw, saved_z=z, activation="gelu", gate=t["gate"], dbias=db, dgate=dgate)
    dres, dy = torch.empty_like(x1), torch.empty_like(y)
    te.te_residual_norm_bwd(dln, dout, x1, mu, rs, gamma, dres, dy, dg, dbeta)
    assert torch.equal(dres, dy)
    want = orc.residual_norm_bwd(f64(dln), f64(dout), f64(x1), f64(mu), f64(rs), f64(gamma))
    within("dy", f64(dy), want["dy"][0], 2.0 ** -17 * want["dy"][1], BF)
    within("dgamma", f64(dg), want["dgamma"][0], 2.0 ** -16 * want["dgamma"][1], F32)
    leaves = [dw, db, dgate, dg, dbeta]
    old = [f64(v) for v in leaves]
    norm = te.te_clip_grad_norm(leaves, 1.0, torch.empty(1, device=DEV))
    length, c = orc.clip(old, 1.0, 1e-6)
    assert abs(norm.item() - length) <= 2.0 ** -19 * length
    for o, v in zip(old, leaves):
        within("clipped", f64(v), o * c, np.abs(o * c) * 2.0 ** -18, v.dtype)

"""Block-scaled operators on the GPU against the float64 oracle (oracle/block_scaled.py).

Packing is held to equality, byte for byte: codes, scales and the zeros that pad a scale tile.
Products: the operands' values are exact, so what differs is the fp32 accumulation.  Each of the
K / 64 tensor-core steps adds a dot product of 64 exact products to an fp32 accumulator; with the
products aligned to the largest of them, a step may lose one unit in the last place per product and
one for the sum: |err| <= (K / 64 + 64) * 2^-23 * sum |a b|, plus half a step of the output's type.
"""

import numpy as np
import pytest
import torch

import fp8_transformer_gb300 as te
from oracle import block as ob
from oracle import block_scaled as bs
from oracle import numerics as nx

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GUARD = 0xA5


def f64(t):
    return t.detach().cpu().double().numpy()


def u8(t):
    return t.detach().cpu().numpy()


def guarded(n):
    """n bytes with a guard of 256 behind them, all set to GUARD."""
    b = torch.full((n + 256,), GUARD, dtype=torch.uint8, device=DEV)
    return b, b[:n]


def draw(rows, cols, dtype, seed=0, std=1.0, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    if spread:  # rows of very different sizes
        x *= 2.0 ** torch.randint(-12, 12, (rows, 1), generator=g)
    return x.to(dtype).to(DEV)


def special(dtype):
    """Zeros, infinities, NaN, subnormals, the type's largest, ties of E2M1 and of the MX scale."""
    x = torch.zeros(40, 96)
    x[1, 3] = float("inf")
    x[2, 40] = float("-inf")
    x[3, 95] = float("nan")
    x[4] = 2.0 ** -133
    x[5] = torch.finfo(dtype).max
    x[6] = torch.tensor([0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, 6.0] * 12)
    x[7] = 6.0 * (1 + 2.0 ** -7)
    x[8, ::32] = 448.0
    x[9, ::32] = 450.0
    x[10] = -0.0
    x[11] = torch.finfo(dtype).tiny
    x[12, 5] = 2.0 ** 100
    x[12, 6] = 2.0 ** -100
    x[32:36] = torch.linspace(-7, 7, 96)
    return x.to(dtype).to(DEV)


def quantize_checked(x, fmt, both, q=None, s=None):
    """te_block_quantize of x against the oracle; returns the buffers."""
    M, N = x.shape
    mp = (M + 31) // 32 * 32
    bufs = {}
    sizes = {"codes": (M, N if fmt == "mxfp8" else N // 2)}
    if both:
        sizes["codes_t"] = (N, mp // 2)
    for k, shape in sizes.items():
        g, v = guarded(shape[0] * shape[1])
        bufs[k] = (g, v.view(*shape))
    for k, (r, c) in {"scales": (M, N), "scales_t": (N, mp)}.items():
        if k == "scales" or both:
            g, v = guarded(te.block_scale_bytes(fmt, r, c))
            bufs[k] = (g, v)
    te.te_block_quantize(x, fmt, q=q, **{k: v[1] for k, v in bufs.items()})
    torch.cuda.synchronize()
    for k, (g, v) in bufs.items():
        assert (g[v.numel():] == GUARD).all(), f"{k}: written past its end"
    xs = f64(x)
    for sfx, src in (("", xs), ("_t", bs.pad_t(xs))):
        if "codes" + sfx not in bufs:
            continue
        c, sc = bs.pack(src, fmt, s)
        got_s, want_s = u8(bufs["scales" + sfx][1]), bs.tile_scales(sc)
        assert np.array_equal(got_s, want_s), (fmt, sfx, np.flatnonzero(got_s != want_s)[:8])
        got_c, want_c = u8(bufs["codes" + sfx][1]), bs.to_bytes(c, fmt)
        assert np.array_equal(got_c, want_c), (fmt, sfx, np.argwhere(got_c != want_c)[:8])
    return {k: v[1] for k, v in bufs.items()}


SHAPES = [(1, 32), (33, 64), (128, 128), (77, 352), (257, 160), (300, 544)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,both", [("mxfp4", False), ("mxfp4", True), ("mxfp8", False)])
def test_mx_packing_is_exact(fmt, both, dtype):
    for i, (m, n) in enumerate(SHAPES):
        quantize_checked(draw(m, n, dtype, seed=i), fmt, both)
    quantize_checked(special(dtype), fmt, both)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("both", [False, True])
def test_nvfp4_packing_is_exact_with_either_scaling(both, dtype):
    for i, (m, n) in enumerate(SHAPES):
        x = draw(m, n, dtype, seed=i, spread=False)
        amax = np.float32(np.abs(f64(x)).max())
        q = te.Quantizer(mode="current")
        s = bs.nv_scale(amax)
        quantize_checked(x, "nvfp4", both, q, s)
        assert q.amax.item() == amax and np.float32(q.scale.item()) == s
        assert np.float32(q.scale_inv.item()) == np.float32(1) / s
        q = te.Quantizer(scale=700.0)  # too large for some blocks: their scales saturate
        quantize_checked(x, "nvfp4", both, q, 700.0)
        assert q.amax.item() == amax and np.float32(q.scale_inv.item()) == np.float32(1) / np.float32(700)
        quantize_checked(x, "nvfp4", both, te.Quantizer.from_tensors(q.scale, q.scale_inv, None), 700.0)
    x = special(dtype)
    quantize_checked(x, "nvfp4", both, te.Quantizer(scale=2.0), 2.0)
    q = te.Quantizer(mode="current")
    quantize_checked(x, "nvfp4", both, q, 1.0)  # an infinite amax: scale 1
    assert q.scale.item() == 1.0
    z = torch.zeros(33, 64, dtype=dtype, device=DEV)
    quantize_checked(z, "nvfp4", both, te.Quantizer(mode="current"), 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nvfp4_zeros_beside_tiny_values(dtype):
    """A tensor so small that s is the largest float and s / scale overflows in its blocks below 1.8e-38:
    their zeros stay zeros, packed along rows, along columns and inside the product."""
    x = torch.zeros(40, 96, device=DEV)
    x[::3, ::5] = 1e-38
    x[1::4, 3::7] = -1.2e-38
    x[7, 3] = 2e-36
    x = x.to(dtype)
    s = bs.nv_scale(np.abs(f64(x)).max())
    assert s == np.finfo(np.float32).max
    quantize_checked(x, "nvfp4", True, te.Quantizer(mode="current"), s)
    quantize_checked(x, "nvfp4", False, te.Quantizer(mode="current"), s)
    w = draw(64, 96, torch.float32, 3, spread=False) * 1e30  # brings the products back into range
    wc, ws = te.block_empty("nvfp4", 64, 96)
    qw, qx = te.Quantizer(mode="current"), te.Quantizer(mode="current")
    te.te_block_quantize(w, "nvfp4", wc, ws, q=qw)
    for rows in (8, 40):  # packed inside the product, and before it
        out = torch.empty(rows, 64, dtype=dtype, device=DEV)
        te.te_dense_fp4_fwd(x[:rows].contiguous(), wc, ws, out, "nvfp4", q=qx, kernel_scale_inv=qw.scale_inv)
        a, b = values(f64(x[:rows]), "nvfp4", s), values(f64(w), "nvfp4", np.float32(qw.scale.item()))
        alpha = float(np.float32(1) / s) * float(np.float32(1) / np.float32(qw.scale.item()))
        want = alpha * (a @ b.T)
        assert (np.abs(f64(out) - want) <= product_bound(a, b, alpha, want, 96, dtype)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N", [(1, 16), (45, 48), (300, 112), (129, 272)])
def test_transposed_alone_with_half_a_block_in_a_row(M, N, fmt, dtype):
    """x^T alone takes rows of x of any multiple of 16, the last block of 32 of them half there."""
    x = draw(M, N, dtype, M, spread=fmt == "mxfp4")
    x[M // 2, N - 1] = -3.0
    mp = (M + 31) // 32 * 32
    gc, ct = guarded(N * mp // 2)
    gs, st = guarded(te.block_scale_bytes(fmt, N, mp))
    q = te.Quantizer(scale=100.0) if fmt == "nvfp4" else None
    te.te_block_quantize(x, fmt, codes_t=ct.view(N, mp // 2), scales_t=st, q=q)
    torch.cuda.synchronize()
    c, s = bs.pack(bs.pad_t(f64(x)), fmt, 100.0)
    assert np.array_equal(u8(ct).reshape(N, -1), bs.to_bytes(c, fmt)) and np.array_equal(u8(st), bs.tile_scales(s))
    assert (gc[ct.numel():] == GUARD).all() and (gs[st.numel():] == GUARD).all()
    if q is not None:
        assert q.amax.item() == x.abs().max().item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_large_tensors_are_packed_like_their_parts(fmt, dtype):
    """Whichever form packs it, a tensor's rows come out as those of a few of them alone (which are held to
    the oracle above)."""
    for M, N in ((4230, 4256), (1800, 4256)):
        x = draw(M, N, dtype, 1, spread=fmt != "nvfp4")
        new = lambda: te.Quantizer(scale=500.0) if fmt == "nvfp4" else None
        codes, scales = te.block_empty(fmt, M, N)
        q = new()
        te.te_block_quantize(x, fmt, codes, scales, q=q)
        per = scales.numel() // ((M + 127) // 128)
        for r in (0, 128 * 7, M // 128 * 128):
            part = x[r:r + 256].contiguous()
            c, s = te.block_empty(fmt, part.shape[0], N)
            te.te_block_quantize(part, fmt, c, s, q=new())
            assert torch.equal(codes[r:r + 256], c)
            assert torch.equal(scales[r // 128 * per:][:s.numel()], s)
        if q is not None:
            assert q.amax.item() == x.abs().max().item()


def test_transposed_alone():
    x = draw(100, 96, torch.bfloat16)
    ct, st = te.block_empty("mxfp4", 96, 128)
    te.te_block_quantize(x, "mxfp4", codes_t=ct, scales_t=st)
    c, s = bs.pack(bs.pad_t(f64(x)), "mxfp4")
    assert np.array_equal(u8(ct), bs.to_bytes(c, "mxfp4")) and np.array_equal(u8(st), bs.tile_scales(s))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_reading_back_is_exact(fmt):
    for i, (m, n) in enumerate(SHAPES + [(40, 96)]):
        x = special(torch.float32) if (m, n) == (40, 96) else draw(m, n, torch.bfloat16, seed=i, spread=fmt != "nvfp4")
        codes, scales = te.block_empty(fmt, m, n)
        q = te.Quantizer(scale=3.0) if fmt == "nvfp4" else None
        te.te_block_quantize(x, fmt, codes, scales, q=q)
        inv = q.scale_inv if q else None
        want = bs.unpack(*bs.pack(f64(x), fmt, 3.0), fmt, np.float32(1) / np.float32(3) if q else None)
        for dt in (torch.float32, torch.bfloat16):
            out = torch.full((m + 1, n), 7.0, dtype=dt, device=DEV)
            te.te_block_dequantize(codes, scales, fmt, out[:m], scale_inv=inv)
            w = nx.bf16_round(want) if dt == torch.bfloat16 else nx.to_f32(want)
            assert np.array_equal(f64(out[:m]), w, equal_nan=True), (fmt, m, n, dt)
            assert (out[m] == 7.0).all()


# ------------------------------------------------------------------------------- products ---


def packed(rows, cols, fmt, seed, scale=64.0):
    """(codes, scales, scale_inv, values) of a random packed tensor."""
    x = draw(rows, cols, torch.bfloat16, seed, spread=fmt != "nvfp4")
    codes, scales = te.block_empty(fmt, rows, cols)
    q = te.Quantizer(scale=scale) if fmt == "nvfp4" else None
    te.te_block_quantize(x, fmt, codes, scales, q=q)
    inv = q.scale_inv if q else None
    c, s = bs.pack(f64(x), fmt, scale)
    return codes, scales, inv, bs.unpack(c, s, fmt), 1.0 if inv is None else inv.item()


def product_bound(a, b, alpha, want, K, dtype):
    return (K / 64 + 64) * 2.0 ** -23 * alpha * (np.abs(a) @ np.abs(b).T) + 2.0 ** -22 * np.abs(want) + \
        HALF_STEP[dtype] * np.abs(want) + 1e-37


def gemm_checked(M, N, K, fmt, bias=None, dtype=torch.bfloat16):
    ca, sa, ia, va, fa = packed(M, K, fmt, 1)
    cb, sb, ib, vb, fb = packed(N, K, fmt, 2, scale=300.0)
    bz = None if bias is None else draw(1, N, bias, seed=3, spread=False)[0].contiguous()
    out = torch.full((M + 1, N), 7.0, dtype=dtype, device=DEV)
    te.te_block_gemm(ca, sa, cb, sb, out[:M], fmt, a_scale_inv=ia, b_scale_inv=ib, bias=bz)
    torch.cuda.synchronize()
    assert te.get_device_status() == 0
    alpha = fa * fb
    want = alpha * (va @ vb.T) + (0 if bz is None else f64(bz))
    err = np.abs(f64(out[:M]) - want)
    tol = product_bound(va, vb, alpha, want, K, dtype) + (0 if bz is None else 2.0 ** -22 * np.abs(f64(bz)))
    assert (out[M] == 7.0).all(), "a row behind the last was written"
    assert (err <= tol).all(), (M, N, K, fmt, float((err / tol).max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [1, 16, 17, 33, 48, 64, 100, 128])
def test_product_of_few_rows(M, fmt):
    gemm_checked(M, 128, 256, fmt)
    gemm_checked(M, 16, 32, fmt, bias=torch.bfloat16)
    gemm_checked(M, 176, 544, fmt, bias=torch.float32, dtype=torch.float32)
    gemm_checked(M, 400, 4096, fmt, bias=torch.bfloat16)
    gemm_checked(M, 1024, 96, fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [129, 256, 300, 513])
def test_product_of_many_rows(M, fmt):
    gemm_checked(M, 256, 256, fmt)
    gemm_checked(M, 16, 32, fmt, bias=torch.bfloat16)
    gemm_checked(M, 272, 544, fmt, bias=torch.float32, dtype=torch.float32)
    gemm_checked(M, 1040, 4128, fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_with_more_tiles_than_sm_pairs(fmt):
    gemm_checked(2100, 3344, 160, fmt, bias=torch.bfloat16)


def test_product_is_the_same_on_every_call():
    for M in (5, 300):
        ca, sa, ia, _, _ = packed(M, 4096, "nvfp4", 1)
        cb, sb, ib, _, _ = packed(512, 4096, "nvfp4", 2)
        outs = [te.te_block_gemm(ca, sa, cb, sb, torch.empty(M, 512, device=DEV), "nvfp4", ia, ib) for _ in range(4)]
        assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_a_bad_block_makes_its_row_nan_and_no_other():
    for M in (7, 200):
        x = draw(M, 512, torch.bfloat16, spread=False)
        x[3, 100] = float("nan")
        for fmt in ("mxfp4", "nvfp4"):
            ca, sa = te.block_empty(fmt, M, 512)
            q = te.Quantizer(scale=64.0) if fmt == "nvfp4" else None
            te.te_block_quantize(x, fmt, ca, sa, q=q)
            cb, sb, _, _, _ = packed(128, 512, fmt, 2)
            out = te.te_block_gemm(ca, sa, cb, sb, torch.empty(M, 128, device=DEV), fmt)
            bad = torch.isnan(out)
            assert bad[3].all() and int(bad.sum()) == 128


# ---------------------------------------------------------------------------- dense layer ---


def values(x, fmt, s):
    c, sc = bs.pack(x, fmt, s)
    return bs.unpack(c, sc, fmt)


@pytest.mark.parametrize("fmt,mode", [("mxfp4", None), ("nvfp4", "current"), ("nvfp4", "delayed")])
@pytest.mark.parametrize("M,K,N,dtype", [(1, 64, 96, torch.bfloat16), (50, 544, 288, torch.float32),
                                         (333, 320, 608, torch.bfloat16), (1, 4096, 320, torch.bfloat16),
                                         (1030, 160, 288, torch.bfloat16), (1100, 96, 64, torch.float32)])
def test_dense_forward_and_backward_together(fmt, mode, M, K, N, dtype):
    """Weights packed once along both axes, the forward keeping x^T, the backward from that."""
    x, dy = draw(M, K, dtype, 1, spread=False), draw(M, N, dtype, 2, spread=False)
    w = draw(K, N, torch.float32, 3, std=0.05, spread=False)
    bias = draw(1, N, dtype, 4, spread=False)[0].contiguous()
    mp = (M + 31) // 32 * 32
    new = (lambda: None) if mode is None else (lambda: te.Quantizer(scale=500.0, mode=mode))
    qw, qx, qg = new(), new(), new()
    wc, ws = te.block_empty(fmt, K, N)
    wct, wst = te.block_empty(fmt, N, K)
    te.te_block_quantize(w, fmt, wc, ws, wct, wst, q=qw)
    xt, xts = te.block_empty(fmt, K, mp)
    out = torch.empty(M, N, dtype=dtype, device=DEV)
    inv = lambda q: None if q is None else q.scale_inv
    te.te_dense_fp4_fwd(x, wct, wst, out, fmt, bias=bias, q=qx, kernel_scale_inv=inv(qw), saved_xt=xt,
                        saved_xt_scales=xts)
    dx = torch.empty(M, K, dtype=dtype, device=DEV)
    dw = torch.empty(K, N, dtype=dtype, device=DEV)
    db = torch.empty(N, dtype=torch.float32, device=DEV)
    te.te_dense_fp4_bwd(dy, wc, ws, xt, xts, dx, dw, fmt, dbias=db, q=qg, kernel_scale_inv=inv(qw),
                        x_scale_inv=inv(qx))
    torch.cuda.synchronize()
    assert te.get_device_status() == 0

    def scale(t):
        return None if mode is None else (bs.nv_scale(np.abs(t).max()) if mode == "current" else np.float32(500))
    xs, ds, wv = f64(x), f64(dy), f64(w)
    sx, sg, sw = scale(xs), scale(ds), scale(wv)
    al = lambda *s: float(np.prod([1.0 if v is None else np.float64(np.float32(1) / np.float32(v)) for v in s]))
    for name, got, a, b, alpha, add in (
            ("out", out, values(xs, fmt, sx), values(wv.T, fmt, sw), al(sx, sw), f64(bias)),
            ("dx", dx, values(ds, fmt, sg), values(wv, fmt, sw), al(sg, sw), 0.0),
            ("dw", dw, values(bs.pad_t(xs), fmt, sx), values(bs.pad_t(ds), fmt, sg), al(sx, sg), 0.0)):
        want = alpha * (a @ b.T) + add
        tol = product_bound(a, b, alpha, want, a.shape[1], dtype) + 2.0 ** -22 * np.abs(add)
        err = np.abs(f64(got) - want)
        assert (err <= tol).all(), (name, float((err / tol).max()))
    # fp32 sums of M values in any order: M roundings at most
    assert (np.abs(f64(db) - ds.sum(0)) <= (M + 4) * 2.0 ** -24 * np.abs(ds).sum(0)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,mode", [("mxfp4", None), ("nvfp4", "current"), ("nvfp4", "delayed")])
@pytest.mark.parametrize("M,K,N", [(1, 32, 16), (1, 4096, 320), (3, 544, 128), (8, 4128, 2064), (9, 96, 400), (17, 1056, 144),
                                   (33, 4096, 256), (40, 288, 2064), (64, 800, 176), (65, 800, 176)])
def test_dense_forward_alone(fmt, mode, dtype, M, K, N):
    """Up to 8 rows the product packs x itself; the row past the last is left as it was, a row with a
    NaN spoils no other, and the result does not vary."""
    x = draw(M, K, dtype, 1, spread=mode is None)
    w = draw(K, N, torch.float32, 3, std=0.05, spread=False)
    bias = draw(1, N, dtype, 4, spread=False)[0].contiguous()
    q = None if mode is None else te.Quantizer(scale=500.0, mode=mode)
    qw = None if mode is None else te.Quantizer(mode="current")
    wct, wst = te.block_empty(fmt, N, K)
    te.te_block_quantize(w, fmt, codes_t=wct, scales_t=wst, q=qw)
    out = torch.full((M + 1, N), 7.0, dtype=dtype, device=DEV)
    call = lambda o: te.te_dense_fp4_fwd(x, wct, wst, o, fmt, bias=bias, q=q,
                                         kernel_scale_inv=None if qw is None else qw.scale_inv)
    call(out[:M])
    again = call(torch.empty(M, N, dtype=dtype, device=DEV))
    torch.cuda.synchronize()
    assert te.get_device_status() == 0
    assert torch.equal(out[:M], again) and (out[M] == 7.0).all()
    xs, wv = f64(x), f64(w)
    sx = sw = None
    alpha = 1.0
    if mode is not None:
        sx = bs.nv_scale(np.abs(xs).max()) if mode == "current" else np.float32(500)
        sw = bs.nv_scale(np.abs(wv).max())
        alpha = float(np.float32(1) / sx) * float(np.float32(1) / sw)
        assert np.float32(q.scale.item()) == sx and np.float32(q.scale_inv.item()) == np.float32(1) / sx
        assert q.amax.item() == np.float32(np.abs(xs).max())
    a, b = values(xs, fmt, sx), values(wv.T, fmt, sw)
    want = alpha * (a @ b.T) + f64(bias)
    tol = product_bound(a, b, alpha, want, K, dtype) + 2.0 ** -22 * np.abs(f64(bias))
    err = np.abs(f64(out[:M]) - want)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])
    if mode != "current":
        x[M - 1, K // 2] = float("nan")
        bad = torch.isnan(call(out[:M]))
        assert bad[M - 1].all() and not bad[:M - 1].any()


def test_dense_without_tokens():
    fmt = "mxfp4"
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    wc, ws = te.block_empty(fmt, 64, 96)
    wct, wst = te.block_empty(fmt, 96, 64)
    xt, xts = te.block_empty(fmt, 64, 0)
    out = torch.empty(0, 96, dtype=torch.bfloat16, device=DEV)
    te.te_dense_fp4_fwd(x, wct, wst, out, fmt, saved_xt=xt, saved_xt_scales=xts)
    dw = torch.full((64, 96), 3.0, dtype=torch.bfloat16, device=DEV)
    db = torch.full((96,), 3.0, device=DEV)
    te.te_dense_fp4_bwd(out, wc, ws, xt, xts, x.clone(), dw, fmt, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


# ---------------------------------------------------------------------------- checkpoints ---

ACTS = ["relu", "gelu", "silu", "swiglu", "geglu", "reglu"]


def ckpt_oracle(act, h, dy):
    """(dx, act(h)) in float64."""
    return ob.act_bwd(dy, h, act), ob.act_fwd(h, act)


def ckpt_checked(act, M, F, dtype, dx_kind, seed=0, mode="delayed", h_std=2.0):
    gated = act in ("swiglu", "geglu", "reglu")
    n_in = 2 * F if gated else F
    h = draw(M, n_in, dtype, seed, std=h_std, spread=False)
    dy = draw(M, F, dtype, seed + 1, spread=False)
    codes, scales = te.block_empty("mxfp8", M, n_in)
    te.te_block_quantize(h, "mxfp8", codes, scales)
    out_dt = {"e4m3": torch.uint8, "same": dtype}[dx_kind]
    dx = torch.zeros(M + 1, n_in, dtype=out_dt, device=DEV)
    a = torch.zeros(M + 1, F, dtype=dtype, device=DEV)
    db = torch.zeros(n_in, device=DEV)
    q = te.Quantizer(scale=16.0, mode=mode) if dx_kind == "e4m3" else None
    te.te_dact_dbias_ckpt(dy, codes, scales, act, dx[:M], dbias=db, act_out=a[:M], q=q)
    torch.cuda.synchronize()
    hv = bs.unpack(*bs.pack(f64(h), "mxfp8"), "mxfp8")
    want, wa = ckpt_oracle(act, hv, f64(dy))
    # the kernels' fp32 arithmetic: hardware exp2 and reciprocal, ~1e-6 relative of each factor; the
    # derivative of gelu and silu cancels near its zero, where the error is relative to its terms
    env = np.abs(f64(dy)) * 1.2 if not gated else np.concatenate(
        [np.abs(f64(dy) * hv[:, F:]) * 1.2, np.abs(f64(dy)) * (np.abs(hv[:, :F]) + 1)], 1)
    err = 1e-5 * env
    assert (np.abs(f64(a[:M]) - wa) <= 1e-5 * np.abs(wa) + 1e-30 + HALF_STEP[dtype] * np.abs(wa)).all()
    assert (np.abs(f64(db) - want.sum(0)) <= err.sum(0) + (M + 8) * 2.0 ** -24 * np.abs(want).sum(0)).all()
    assert (dx[M] == 0).all() and (a[M] == 0).all()
    if dx_kind == "same":
        assert (np.abs(f64(dx[:M]) - want) <= err + HALF_STEP[dtype] * np.abs(want)).all()
    else:
        amax = np.abs(want).max()
        assert abs(q.amax.item() - amax) <= err.max()
        s = float(q.scale.item())
        if mode == "current":
            assert s == nx.compute_scale(q.amax.item())[0]
        got = nx.e4m3_decode(u8(dx[:M]))
        lo, hi = (nx.e4m3_decode(nx.e4m3_encode((want + k * err) * s)) for k in (-1, 1))
        assert ((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi))).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_from_checkpoint(act, dtype):
    ckpt_checked(act, 1, 32, dtype, "same")
    ckpt_checked(act, 130, 288, dtype, "same", seed=5)
    ckpt_checked(act, 300, 544, dtype, "e4m3", seed=7)
    ckpt_checked(act, 77, 160, dtype, "e4m3", seed=9, mode="current")


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu", "geglu"])
def test_gradient_from_checkpoint_far_from_zero(act):
    """Pre-activations far out: the activation and its derivative reach their limits, never NaN."""
    M, F = 4, 64
    n_in = 2 * F if act in ("swiglu", "geglu") else F
    big = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 1e4, -1e4, 1e20, -1e20, 1e30, -1e30] * 11)[:n_in]
    h = big.sort().values.repeat(M, 1).to(DEV)
    h[1] = h[1].flip(0)
    dy = torch.ones(M, F, device=DEV)
    codes, scales = te.block_empty("mxfp8", M, n_in)
    te.te_block_quantize(h, "mxfp8", codes, scales)
    dx, a = torch.empty(M, n_in, device=DEV), torch.empty(M, F, device=DEV)
    te.te_dact_dbias_ckpt(dy, codes, scales, act, dx, act_out=a)
    hv = bs.unpack(*bs.pack(f64(h), "mxfp8"), "mxfp8")
    with np.errstate(all="ignore"):
        g = hv[:, :F]
        s = 1 / (1 + np.exp(-g)) if act in ("silu", "swiglu") else 1 / (1 + np.exp(-2 * 0.7978845608028654 * (g + 0.044715 * g ** 3)))
        y = np.where(np.isfinite(g * s), g * s, 0.0)
        lin = hv[:, F:] if n_in > F else 1.0
        wa = y * lin
    assert torch.isfinite(dx).all()
    fin = np.abs(wa) < 3e38
    assert (np.abs(f64(a) - wa)[fin] <= 1e-5 * np.abs(wa)[fin] + 1e-30).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("act", ACTS)
def test_gradient_from_a_bad_block_is_nan(act, kind):
    """A NaN or an infinity makes its block NaN: activation, gradient and column sums say so, and no other
    block does."""
    M, F = 130, 96
    gated = act in ("swiglu", "geglu", "reglu")
    n_in = 2 * F if gated else F
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    h, dy = draw(M, n_in, dtype, 1, spread=False), draw(M, F, dtype, 2, spread=False)
    dy[dy == 0] = 1.0
    h[3, 40] = float("nan")    # block 1 of row 3
    h[129, 95] = float("inf")  # block 2 of row 129
    h[70, 0] = float("-inf")   # block 0 of row 70
    bad = torch.zeros(M, n_in, dtype=torch.bool, device=DEV)  # of h
    for r, c in ((3, 32), (129, 64), (70, 0)):
        bad[r, c:c + 32] = True
    if gated:
        h[5, F + 33] = float("nan")  # the linear half alone
        bad[5, F + 32:F + 64] = True
    codes, scales = te.block_empty("mxfp8", M, n_in)
    te.te_block_quantize(h, "mxfp8", codes, scales)
    dx = torch.empty(M, n_in, dtype=torch.uint8 if kind == "e4m3" else dtype, device=DEV)
    a, db = torch.empty(M, F, dtype=dtype, device=DEV), torch.empty(n_in, device=DEV)
    q = te.Quantizer(scale=16.0) if kind == "e4m3" else None
    te.te_dact_dbias_ckpt(dy, codes, scales, act, dx, dbias=db, act_out=a, q=q)
    dx = dx.view(torch.float8_e4m3fn).float() if kind == "e4m3" else dx.float()
    # act(gate) * lin and both gradients but the linear half's, dy * act(gate), depend on the linear half
    of_act = bad[:, :F] | bad[:, F:] if gated else bad
    of_dx = torch.cat([of_act, bad[:, :F]], 1) if gated else bad
    assert torch.equal(torch.isnan(a), of_act)
    assert torch.equal(torch.isnan(dx), of_dx)
    assert torch.equal(torch.isnan(db), of_dx.any(0))
    assert torch.isfinite(dx[~of_dx]).all() and torch.isfinite(a[~of_act]).all()
    if q is not None:
        assert np.isfinite(q.amax.item()) and q.amax.item() > 0


def test_gradient_from_checkpoint_by_differences():
    """dx is the slope of sum(dy * act(h)) at the checkpointed h (central differences, float64)."""
    for act in ("gelu", "silu", "swiglu", "geglu"):
        M, F = 3, 32
        n_in = 2 * F if act in ("swiglu", "geglu") else F
        h, dy = draw(M, n_in, torch.float32, 1, spread=False), draw(M, F, torch.float32, 2, spread=False)
        codes, scales = te.block_empty("mxfp8", M, n_in)
        te.te_block_quantize(h, "mxfp8", codes, scales)
        dx = torch.empty(M, n_in, device=DEV)
        te.te_dact_dbias_ckpt(dy, codes, scales, act, dx)
        hv, e = bs.unpack(*bs.pack(f64(h), "mxfp8"), "mxfp8"), 1e-5
        for i, j in ((0, 0), (1, n_in - 1), (2, n_in // 2), (2, 5)):
            d = np.zeros_like(hv)
            d[i, j] = e
            slope = ((f64(dy) * (ob.act_fwd(hv + d, act) - ob.act_fwd(hv - d, act))).sum()) / (2 * e)
            assert abs(slope - dx[i, j].item()) <= 1e-5 * max(1.0, abs(slope)) + 1e-8


# ---------------------------------------------------------------- streams, graphs, layout ---


def test_captured_and_replayed_on_other_inputs():
    M, K, N, fmt = 9, 512, 256, "nvfp4"
    xs = [draw(M, K, torch.bfloat16, s, spread=False) for s in (1, 2)]
    cb, sb, ib, _, _ = packed(N, K, fmt, 5)
    q = te.Quantizer(mode="current")
    ws = torch.empty(te.workspace_size(te.binding.TE_OP_DENSE_FP4_FWD, M, K, N), dtype=torch.uint8, device=DEV)
    eager = [te.te_dense_fp4_fwd(x, cb, sb, torch.empty(M, N, dtype=torch.bfloat16, device=DEV), fmt, q=q,
                                 kernel_scale_inv=ib) for x in xs]
    x, out = xs[0].clone(), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        te.te_dense_fp4_fwd(x, cb, sb, out, fmt, q=q, kernel_scale_inv=ib, workspace=ws)
    for k in (0, 1, 0):
        x.copy_(xs[k])
        g.replay()
        assert torch.equal(out, eager[k])


def test_on_another_stream_without_a_workspace_of_its_own():
    M, K, N, fmt = 200, 1024, 512, "mxfp4"
    x = draw(M, K, torch.bfloat16, 1)
    cb, sb, _, _, _ = packed(N, K, fmt, 2)
    want = te.te_dense_fp4_fwd(x, cb, sb, torch.empty(M, N, dtype=torch.bfloat16, device=DEV), fmt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    for o in outs:
        te.te_dense_fp4_fwd(x, cb, sb, o, fmt, stream=s)
        torch.empty(M * K, dtype=torch.uint8, device=DEV).fill_(255)  # would land in a workspace freed too early
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in outs)


def test_nothing_is_kept_for_a_stream_made_elsewhere():
    M, K, N, fmt = 20, 512, 256, "mxfp4"
    x = draw(M, K, torch.bfloat16, 1)
    cb, sb, _, _, _ = packed(N, K, fmt, 2)
    want = te.te_dense_fp4_fwd(x, cb, sb, torch.empty(M, N, dtype=torch.bfloat16, device=DEV), fmt)
    pooled = torch.cuda.Stream()
    torch.cuda.synchronize()
    te.binding._small.kept.clear()  # the pool may have handed this stream out before
    kept = lambda: {h for _, h in te.binding._small.kept}
    for stream, lasts in ((torch.cuda.ExternalStream(pooled.cuda_stream), False), (pooled, True)):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            outs = [te.te_dense_fp4_fwd(x, cb, sb, torch.empty(M, N, dtype=torch.bfloat16, device=DEV), fmt) for _ in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(want, o) for o in outs)
        assert (pooled.cuda_stream in kept()) == lasts


def dense_backward_inputs(fmt, M, K, N, seeds):
    """(calls, packed weights and x^T) of te_dense_fp4_bwd; calls(i, **kw) on dy number i -> dx, dw, db."""
    dys = [draw(M, N, torch.bfloat16, s, spread=False) for s in seeds]
    kc, ks, ik, _, _ = packed(K, N, fmt, 21)
    xt, xts, ix, _, _ = packed(K, (M + 31) // 32 * 32, fmt, 22)

    def call(dy, q, out=None, **kw):
        dx, dw, db = out or (torch.empty(M, K, dtype=torch.bfloat16, device=DEV),
                             torch.empty(K, N, dtype=torch.bfloat16, device=DEV), torch.empty(N, device=DEV))
        te.te_dense_fp4_bwd(dy, kc, ks, xt, xts, dx, dw, fmt, dbias=db, q=q, kernel_scale_inv=ik, x_scale_inv=ix, **kw)
        return dx, dw, db
    return dys, call


@pytest.mark.parametrize("fmt,mode", [("mxfp4", None), ("nvfp4", "current"), ("nvfp4", "delayed")])
@pytest.mark.parametrize("M", [20, 300])
def test_dense_backward_captured_and_replayed_on_other_inputs(fmt, mode, M):
    """With a workspace of the caller's and with the graph's own."""
    K, N = 288, 416
    dys, call = dense_backward_inputs(fmt, M, K, N, (1, 2))
    new = lambda: None if mode is None else te.Quantizer(scale=300.0, mode=mode)
    want = [call(dy, new()) for dy in dys]
    ws = torch.empty(te.workspace_size(te.binding.TE_OP_DENSE_FP4_BWD, M, K, N), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for kw in (dict(workspace=ws), dict()):
        dy, q = dys[0].clone(), new()
        out = tuple(torch.empty_like(t) for t in want[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(dy, q, out, **kw)
        for k in (0, 1, 0):
            dy.copy_(dys[k])
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want[k])), (kw.keys(), k)
    assert te.get_device_status() == 0


def test_dense_backward_on_another_stream():
    """On the current stream and on one that is passed, whose workspace lasts until that stream is past it."""
    M, K, N, fmt = 260, 544, 512, "mxfp4"
    dys, call = dense_backward_inputs(fmt, M, K, N, (1, 2))
    want = [call(dy, None) for dy in dys]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [[tuple(torch.empty_like(t) for t in want[0]) for _ in range(8)] for _ in range(2)]
    for i, o in enumerate(outs[0]):
        call(dys[i % 2], None, o, stream=s)
        torch.empty(M * N, dtype=torch.uint8, device=DEV).fill_(255)  # would land in a workspace freed too early
    with torch.cuda.stream(s):
        for i, o in enumerate(outs[1]):
            call(dys[i % 2], None, o)
    torch.cuda.synchronize()
    for o in outs:
        for i, got in enumerate(o):
            assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2])), i


def test_chains_through_the_same_buffers_without_waits():
    """Each kernel may start before the one whose output it reads has ended: with buffers that take other
    values every time, nothing of the time before is read."""
    M, F, act = 300, 544, "swiglu"
    hs = [draw(M, 2 * F, torch.bfloat16, s, spread=False) for s in (1, 2, 3)]
    dy = draw(M, F, torch.bfloat16, 4, spread=False)
    codes, scales = te.block_empty("mxfp8", M, 2 * F)

    def gradient(i):
        dx, a = torch.empty(M, 2 * F, dtype=torch.uint8, device=DEV), torch.empty(M, F, dtype=torch.bfloat16, device=DEV)
        db, q = torch.empty(2 * F, device=DEV), te.Quantizer(scale=16.0)
        te.te_block_quantize(hs[i], "mxfp8", codes, scales)
        te.te_dact_dbias_ckpt(dy, codes, scales, act, dx, dbias=db, act_out=a, q=q)
        return dx, a, db, q.amax

    T, K, N, fmt = 4, 1024, 768, "mxfp4"  # two layers of four tokens, each packing its input itself
    xs = [draw(T, K, torch.bfloat16, s, spread=False) for s in (5, 6, 7)]
    c1, s1, _, _, _ = packed(N, K, fmt, 8)
    c2, s2, _, _, _ = packed(K, N, fmt, 9)
    mid, bias = torch.empty(T, N, dtype=torch.bfloat16, device=DEV), draw(1, K, torch.bfloat16, 10, spread=False)[0]

    def layers(i):
        out = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
        te.te_dense_fp4_fwd(xs[i], c1, s1, mid, fmt)
        return (te.te_dense_fp4_fwd(mid, c2, s2, out, fmt, bias=bias),)

    for f in (gradient, layers):
        want = []
        for i in range(3):
            want.append(f(i))
            torch.cuda.synchronize()
        got = [f(i % 3) for i in range(60)]
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert all(torch.equal(u, v) for u, v in zip(g, want[i % 3])), (f.__name__, i)


def test_checkpoint_gradients_on_two_streams_at_once():
    """Each stream's calls sum their columns in a workspace of that stream's."""
    M, F, act = 1000, 1024, "geglu"
    hs = [draw(M, 2 * F, torch.bfloat16, s, spread=False) for s in (1, 2)]
    dy = draw(M, F, torch.bfloat16, 3, spread=False)
    packs = [te.block_empty("mxfp8", M, 2 * F) for _ in hs]
    for h, p in zip(hs, packs):
        te.te_block_quantize(h, "mxfp8", *p)

    def call(i):
        dx, db = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=DEV), torch.empty(2 * F, device=DEV)
        te.te_dact_dbias_ckpt(dy, *packs[i], act, dx, dbias=db)
        return dx, db
    want = [call(i) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in hs]
    got = []
    for n in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, call(i)))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(u, v) for u, v in zip(g, want[i]))


def test_two_host_threads_at_once():
    """Calls of two threads on one stream interleave; each has a workspace of its own."""
    import threading
    fmt, M, K, N = "nvfp4", 40, 1024, 256
    cb, sb, ib, _, _ = packed(N, K, fmt, 5)
    xs = [draw(M, K, torch.bfloat16, s, spread=False) for s in (1, 2)]
    qs = [te.Quantizer(mode="current") for _ in xs]
    call = lambda i, o: te.te_dense_fp4_fwd(xs[i], cb, sb, o, fmt, q=qs[i], kernel_scale_inv=ib)
    want = [call(i, torch.empty(M, N, dtype=torch.bfloat16, device=DEV)) for i in (0, 1)]
    outs = [[torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(100)] for _ in xs]

    def work(i):
        for o in outs[i]:
            call(i, o)
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are what they are alone."""
    M, N = 66000, 32768 + 512
    x = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    for r in range(0, M, 8000):
        x[r:r + 8000].normal_()
    last = slice(M - 80, M)
    tile = slice(M // 128 * 128, M)
    for fmt in ("mxfp8", "mxfp4"):
        codes, scales = te.block_empty(fmt, M, N)
        ct = st = None
        if fmt == "mxfp4":
            mp = (M + 31) // 32 * 32
            ct, st = te.block_empty(fmt, N, mp)
        te.te_block_quantize(x, fmt, codes, scales, ct, st)
        own = x[tile].contiguous()
        c2, s2 = te.block_empty(fmt, own.shape[0], N)
        te.te_block_quantize(own, fmt, c2, s2)
        assert torch.equal(codes[tile], c2)
        assert torch.equal(scales[-s2.numel():], s2)
        back = te.te_block_dequantize(codes, scales, fmt, torch.empty_like(x))
        b2 = te.te_block_dequantize(c2, s2, fmt, torch.empty_like(own))
        assert torch.equal(back[tile], b2)
        if fmt == "mxfp8":
            dy = back  # any values
            dx, a = torch.empty_like(x), torch.empty_like(x)
            te.te_dact_dbias_ckpt(dy, codes, scales, "silu", dx, act_out=a)
            d2, a2 = torch.empty_like(own), torch.empty_like(own)
            te.te_dact_dbias_ckpt(dy[tile].contiguous(), c2, s2, "silu", d2, act_out=a2)
            assert torch.equal(dx[tile], d2) and torch.equal(a[tile], a2)
            del dx, a, dy
        else:
            t2, u2 = te.block_empty(fmt, 128, mp)
            te.te_block_quantize(x[:, -128:].contiguous(), fmt, codes_t=t2, scales_t=u2)
            assert torch.equal(ct[-128:], t2)
        del back
    # a product with that many outputs: columns of a small one
    K = 64
    A, B = te.block_empty("mxfp4", M, K), te.block_empty("mxfp4", N, K)
    te.te_block_quantize(draw(M, K, torch.bfloat16, 1, spread=False), "mxfp4", *A)
    te.te_block_quantize(draw(N, K, torch.bfloat16, 2, spread=False), "mxfp4", *B)
    te.te_block_gemm(*A, *B, x, "mxfp4")
    small = torch.empty(M, 128, dtype=torch.bfloat16, device=DEV)
    te.te_block_gemm(*A, B[0][-128:].contiguous(), B[1][-512:].contiguous(), small, "mxfp4")
    assert torch.equal(x[:, -128:][last], small[last])
    assert te.get_device_status() == 0


def test_a_checkpoint_of_more_than_2_to_the_30_columns():
    """Its scales take 4 bytes a column: offsets past 32 bits within one row of tiles."""
    N = (1 << 30) + 256
    x = torch.zeros(1, N, dtype=torch.bfloat16, device=DEV)
    x[0, :256], x[0, -256:], x[0, N // 2:N // 2 + 256] = 1.0, 8.0, 2.0 ** 20
    codes, scales = te.block_empty("mxfp8", 1, N)
    te.te_block_quantize(x, "mxfp8", codes, scales)
    dx, a = torch.empty_like(x), torch.empty_like(x)
    te.te_dact_dbias_ckpt(x, codes, scales, "relu", dx, act_out=a)
    assert torch.equal(a, x) and torch.equal(dx, x)
    assert te.get_device_status() == 0


def test_tensors_the_binding_refuses():
    x = draw(32, 64, torch.bfloat16)
    c, s = te.block_empty("mxfp4", 32, 64)
    with pytest.raises(ValueError, match="contiguous"):
        te.te_block_quantize(draw(64, 32, torch.bfloat16).t(), "mxfp4", c, s)
    with pytest.raises(ValueError, match="codes: shape"):
        te.te_block_quantize(x, "mxfp4", c[:, :16].contiguous(), s)
    with pytest.raises(ValueError, match="scales"):
        te.te_block_quantize(x, "mxfp4", c, s[:100])
    with pytest.raises(ValueError, match="q:"):
        te.te_block_quantize(x, "nvfp4", c, te.block_empty("nvfp4", 32, 64)[1])
    with pytest.raises(ValueError, match="dtype"):
        te.te_block_quantize(x.half(), "mxfp4", c, s)
    with pytest.raises((ValueError, RuntimeError)):
        te.te_block_quantize(x.cpu(), "mxfp4", c, s)
    with pytest.raises(te.TEError):  # a row length that is not whole blocks
        te.te_block_quantize(draw(4, 48, torch.bfloat16), "mxfp4", *te.block_empty("mxfp4", 4, 48))
    with pytest.raises(te.TEError):  # 8-bit codes do not go into the 4-bit product
        e, f = te.block_empty("mxfp8", 32, 64)
        te.te_block_gemm(e, f, e, f, torch.empty(32, 32, device=DEV), "mxfp8")


def test_scales_without_their_codes_are_refused():
    """They would be left as they were."""
    x, (c, s) = draw(32, 64, torch.bfloat16), te.block_empty("mxfp4", 32, 64)
    ct, st = te.block_empty("mxfp4", 64, 32)
    with pytest.raises(ValueError, match="scales_t: given without"):
        te.te_block_quantize(x, "mxfp4", c, s, scales_t=st)
    with pytest.raises(ValueError, match="scales: given without"):
        te.te_block_quantize(x, "mxfp4", scales=s, codes_t=ct, scales_t=st)
    with pytest.raises(ValueError, match="saved_xt_scales: given without"):
        te.te_dense_fp4_fwd(x, c, s, torch.empty(32, 32, dtype=torch.bfloat16, device=DEV), "mxfp4", saved_xt_scales=st)

"""The oracle's block-scaled formats against brute force, torch's E4M3 cast and their own bounds."""

import numpy as np
import pytest
import torch

from oracle import block_scaled as bs
from oracle import numerics as nx


def test_e2m1_nearest_even_by_brute_force():
    v = np.concatenate([np.linspace(-7, 7, 2801), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e9, -0.0]])
    got = bs.e2m1_encode(v)
    for x, c in zip(v, got):
        d = np.abs(bs.E2M1 - min(abs(x), 6.0))
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
        assert c == want | (int(np.signbit(x)) << 3), x
    assert np.array_equal(bs.e2m1_decode(np.arange(8)), bs.E2M1)
    assert np.signbit(bs.e2m1_decode(np.array([8])))[0]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_round_trip_within_half_a_step_of_the_block(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((37, 96)).astype(np.float32) * 2.0 ** rng.integers(-20, 20, (37, 1))
    x[5] = 0.0
    x = x.astype(np.float32).astype(np.float64)
    s = bs.nv_scale(np.abs(x[7]).max()) if fmt == "nvfp4" else None
    rows = slice(7, 8) if fmt == "nvfp4" else slice(None)
    x = x[rows]
    c, sc = bs.pack(x, fmt, s)
    y = bs.unpack(c, sc, fmt, None if s is None else np.float32(1) / s)
    a = np.abs(x).reshape(x.shape[0], -1, bs.BLOCK[fmt]).max(-1).repeat(bs.BLOCK[fmt], -1)
    # the widest step is 2 of 6 (E2M1; a block's scale, rounded up to a power of two, doubles it) or 32
    # of 448; NVFP4's block scale is itself off by up to 1/16
    bound = {"mxfp4": a / 3, "nvfp4": a / 6 * 1.13 + a / 16, "mxfp8": a / 14}[fmt]
    assert (np.abs(x - y) <= bound + 1e-300).all()


def test_mx_scale_is_the_smallest_power_of_two_that_does_not_saturate():
    for fmt in ("mxfp4", "mxfp8"):
        top = bs.TOP[fmt]
        for a in (top, np.nextafter(np.float32(top), np.float32(1e9)), top * 0.5, 1.0, 3.0, 2.0 ** -126, 2.0 ** -149,
                  3.3e38):
            x = np.zeros((1, 32))
            x[0, 3] = -float(np.float32(a))
            _, s = bs.pack(x, fmt)
            f = bs.e8m0_decode(s)[0, 0]
            assert abs(x[0, 3]) / f <= top and (s[0, 0] == 0 or abs(x[0, 3]) / (f / 2) > top)


def test_a_block_with_inf_or_nan_reads_as_nan_and_no_other_does():
    for fmt in ("mxfp4", "nvfp4", "mxfp8"):
        x = np.ones((2, 96))
        x[0, 1], x[1, 40] = np.inf, np.nan
        c, s = bs.pack(x, fmt, 2688.0)
        y = bs.unpack(c, s, fmt, 1 / 2688.0)
        n = bs.BLOCK[fmt]
        assert np.isnan(y[0, :n]).all() and np.isnan(y[1, 40 // n * n:40 // n * n + n]).all()
        assert np.isnan(y).sum() == 2 * n


def test_bytes_and_tiles_there_and_back():
    rng = np.random.default_rng(2)
    c = rng.integers(0, 16, (5, 64)).astype(np.uint8)
    assert np.array_equal(bs.from_bytes(bs.to_bytes(c, "mxfp4"), "mxfp4"), c)
    assert bs.to_bytes(np.array([[3, 9]], np.uint8), "mxfp4")[0, 0] == 0x93
    s = rng.integers(1, 255, (300, 7)).astype(np.uint8)
    t = bs.tile_scales(s)
    assert t.size == 3 * 2 * 512 and np.array_equal(bs.untile_scales(t, 300, 7), s)
    assert np.count_nonzero(t) == s.size
    assert t[(2 * 2 + 1) * 512 + 8 * 16 + 1 * 4 + 2] == s[256 + 32 + 8, 6]


def test_mxfp8_codes_are_torchs_cast_of_the_scaled_values():
    x = torch.randn(8, 64, generator=torch.Generator().manual_seed(3))
    c, s = bs.pack(x.double().numpy(), "mxfp8")
    f = torch.from_numpy(bs.e8m0_decode(s)).float().repeat_interleave(32, 1)
    assert np.array_equal(c, (x / f).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert nx.e4m3_decode(c).max() <= 448


def test_a_zero_stays_zero_where_the_factor_overflows():
    """s / scale past the largest float: that float in its place, so that 0 times it is 0."""
    x = np.zeros((1, 48))
    x[0, 1], x[0, 17], x[0, 40] = 2e-36, -1e-38, 1.2e-38
    s = bs.nv_scale(2e-36)
    assert s == np.finfo(np.float32).max
    c, sc = bs.pack(x, "nvfp4", s)
    assert (sc > 0).all() and np.array_equal(np.flatnonzero(c), [1, 17, 40])
    assert c[0, 17] == 8 + 5 and c[0, 40] == 6  # -1e-38 * 3.4e38 = -3.4 -> -3, 4.08 -> 4

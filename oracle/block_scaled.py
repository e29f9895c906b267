"""Block-scaled formats (MXFP4, NVFP4, MXFP8) in float64, from the definitions in te_gb300.h.

Test infrastructure, never product code (see ``oracle/__init__.py``).  A tensor [rows, cols] is
packed along its columns: every block of neighbours shares one scale.  Where a definition rounds
to fp32 on the way (NVFP4's tensor scale), so does this.
"""

from __future__ import annotations

import numpy as np

from . import numerics as nx

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32}
TOP = {"mxfp4": 6.0, "nvfp4": 6.0, "mxfp8": 448.0}


def e2m1_encode(v) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, saturating; the sign is bit 3."""
    a = np.minimum(np.abs(np.asarray(v, np.float64)), 6.0)
    hi = np.searchsorted(E2M1, a, side="left")          # first grid point >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes, np.int64)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def nv_scale(amax) -> np.float32:
    """fp32 tensor scale of NVFP4: 2688 / amax."""
    amax = np.float32(amax)
    if not np.isfinite(amax) or amax == 0:
        return np.float32(1.0)
    with np.errstate(over="ignore"):
        s = np.float32(2688.0) / amax
    return s if np.isfinite(s) else np.float32(np.finfo(np.float32).max)


def e8m0_decode(b) -> np.ndarray:
    b = np.asarray(b, np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.minimum(b, 254) - 127))


def pack(x, fmt, s=None):
    """(codes, scales [rows, blocks]) of fp32 / bf16 values x (float64 array holding them); codes
    one to an element."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK[fmt], BLOCK[fmt])
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    if fmt == "nvfp4":
        s32 = np.float32(s)
        with np.errstate(over="ignore"):
            t = (amax.astype(np.float32) * s32) / np.float32(6.0)
        sb = nx.e4m3_encode(t.astype(np.float64))
        sf = nx.e4m3_decode(sb).astype(np.float32)
        with np.errstate(divide="ignore", over="ignore"):
            e = np.where(sf > 0, s32 / np.where(sf > 0, sf, np.float32(1)), np.float32(0))
        e = np.where(np.isposinf(e), np.finfo(np.float32).max, e)  # so that a zero stays a zero
        with np.errstate(over="ignore", invalid="ignore"):
            v = (b.astype(np.float32) * e[..., None].astype(np.float32)).astype(np.float64)
        scales = np.where(bad, 0x7F, sb)
    else:
        m, ex = np.frexp(amax / TOP[fmt])   # amax / top = m 2^ex, m in [0.5, 1)
        p = np.where(m == 0.5, ex - 1, ex)  # smallest power of two at or above it
        p = np.where(amax == 0, -127, np.maximum(p, -127))
        v = b / np.ldexp(1.0, p)[..., None]
        scales = np.where(bad, 255, p + 127)
    v = np.where(bad[..., None], 0.0, v).reshape(rows, cols)
    codes = nx.e4m3_encode(v) if fmt == "mxfp8" else e2m1_encode(v)
    return codes, scales.astype(np.uint8)


def unpack(codes, scales, fmt, s_inv=None):
    """fp32 values (as float64) of one-to-an-element codes and [rows, blocks] scales."""
    rows, cols = codes.shape
    v = nx.e4m3_decode(codes) if fmt == "mxfp8" else e2m1_decode(codes)
    f = nx.e4m3_decode(scales) if fmt == "nvfp4" else e8m0_decode(scales)
    v = (v.reshape(rows, cols // BLOCK[fmt], BLOCK[fmt]) * f[..., None]).reshape(rows, cols)
    if s_inv is not None:
        v = (v.astype(np.float32) * np.float32(s_inv)).astype(np.float64)
    return v


def to_bytes(codes, fmt):
    """One-to-an-element codes -> the stored bytes (two E2M1 codes to a byte, the earlier lower)."""
    return codes if fmt == "mxfp8" else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def from_bytes(b, fmt):
    if fmt == "mxfp8":
        return b
    return np.stack((b & 15, b >> 4), -1).reshape(b.shape[0], -1)


def tile_scales(s):
    """[rows, blocks] -> the stored bytes: tiles of 128 rows x 4 blocks, zeros where there is none."""
    rows, nb = s.shape
    rt, g = -(-rows // 128), -(-nb // 4)
    out = np.zeros((rt * g, 512), np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[(r // 128) * g + b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s[r, b]
    return out.reshape(-1)


def untile_scales(t, rows, nb):
    g = -(-nb // 4)
    t = np.asarray(t).reshape(-1)
    r, b = np.arange(rows)[:, None], np.arange(nb)[None, :]
    return t[((r // 128) * g + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def pad_t(x):
    """x^T with the rows of x filled up to a multiple of 32 with zeros."""
    m, n = x.shape
    t = np.zeros((n, (m + 31) // 32 * 32))
    t[:, :m] = x.T
    return t

"""What is measured of the block-scaled operators: 4-bit quantisation and products, and 8-bit
activation checkpoints with the backward pass that reads them.

Formats (a block is a run of neighbours along the packed axis that share one scale):
  mxfp4  E2M1 codes, two a byte (the lower half first), 32 to a block, E8M0 scale (a power of two)
  nvfp4  E2M1 codes, 16 to a block, E4M3 scale, and one fp32 scale for the tensor
  mxfp8  E4M3 codes, 32 to a block, E8M0 scale
Scales lie in tiles of 128 rows x 4 blocks (512 bytes): row r, block b of a tile is byte
(r % 32) * 16 + (r / 32) * 4 + b; tiles go along a row of tiles first; what pads a tile is zero.
"""

import math

import torch

own = False

_BLOCK = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32}
_TOP = {"mxfp4": 6.0, "nvfp4": 6.0, "mxfp8": 448.0}
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_GATED = ("swiglu", "geglu", "reglu")
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------------------- the cases ---


def listed():
    return [
        # the hidden states of 16 sequences that generate, packed before a 4-bit product
        dict(name="quantize decode batch", op="quantize", fmt="mxfp4", dtype="bf16", rows=16, cols=4096,
             both=False, scaling="none"),
        # the gradient of a gated feed-forward layer, packed along both axes for its two products;
        # the token count is ragged
        dict(name="quantize gradient both ways", op="quantize", fmt="nvfp4", dtype="bf16", rows=8190,
             cols=14336, both=True, scaling="current"),
        # fp32 master weights of a gated up projection, packed for the forward and the backward
        dict(name="quantize master weights", op="quantize", fmt="mxfp4", dtype="f32", rows=4096,
             cols=28672, both=True, scaling="none"),
        # a feed-forward layer's pre-activation, stored as an 8-bit checkpoint and read back
        dict(name="checkpoint store and read", op="quantize", fmt="mxfp8", dtype="bf16", rows=4095,
             cols=16384, both=False, scaling="none"),
        # one token through a gated up projection
        dict(name="dense one token", op="dense_fwd", fmt="mxfp4", dtype="bf16", M=1, K=4096, N=28672,
             bias=False, scaling="none"),
        # an odd batch of tokens through the down projection, scales from earlier steps
        dict(name="dense 33 tokens", op="dense_fwd", fmt="nvfp4", dtype="bf16", M=33, K=14336, N=4096,
             bias=True, scaling="delayed"),
        # a prompt through the QKV projection, this call's scale
        dict(name="dense prompt", op="dense_fwd", fmt="nvfp4", dtype="bf16", M=1000, K=8192, N=24576,
             bias=True, scaling="current"),
        # a training batch through the gated up projection
        dict(name="dense training forward", op="dense_fwd", fmt="mxfp4", dtype="bf16", M=8192, K=4096,
             N=28672, bias=False, scaling="none"),
        # the two products of a feed-forward layer's backward pass, ragged token count
        dict(name="dense training backward", op="dense_bwd", fmt="mxfp4", dtype="bf16", M=4100, K=4096,
             N=16384, scaling="none"),
        # the backward of gelu from 8-bit checkpoints at full size, the activation recomputed
        dict(name="checkpoint backward gelu", op="ckpt_bwd", act="gelu", dtype="bf16", M=16384, F=16384,
             dx="bf16", act_out=True),
        # the gated backward of a short batch, its gradient stored in E4M3
        dict(name="checkpoint backward swiglu", op="ckpt_bwd", act="swiglu", dtype="bf16", M=777,
             F=14336, dx="e4m3", act_out=True),
        # a tiny fp32 layer
        dict(name="checkpoint backward tiny", op="ckpt_bwd", act="silu", dtype="f32", M=64, F=512,
             dx="f32", act_out=True),
    ]


def _size(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["quantize", "quantize", "dense_fwd", "dense_fwd", "dense_bwd", "ckpt_bwd", "ckpt_bwd"])
    if op == "quantize":
        fmt = rng.choice(["mxfp4", "nvfp4", "mxfp8"])
        both = fmt != "mxfp8" and rng.random() < 0.5
        return dict(op=op, fmt=fmt, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=_size(rng, 1, 8192),
                    cols=_size(rng, 32, 12288, 32), both=both,
                    scaling=rng.choice(["current", "delayed"]) if fmt == "nvfp4" else "none")
    if op in ("dense_fwd", "dense_bwd"):
        fmt = rng.choice(["mxfp4", "nvfp4"])
        scaling = rng.choice(["current", "delayed"]) if fmt == "nvfp4" else "none"
        K = _size(rng, 128, 14336, 32)
        N = _size(rng, 128, 24576, 32)
        c = dict(op=op, fmt=fmt, dtype="bf16", M=_size(rng, 1, 4096), K=K, N=N, scaling=scaling)
        if op == "dense_fwd":
            c["bias"] = rng.random() < 0.5
        return c
    act = rng.choice(["relu", "gelu", "silu", "swiglu", "geglu", "reglu"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    return dict(op=op, act=act, dtype=dtype, M=_size(rng, 1, 8192), F=_size(rng, 32, 14336, 32),
                dx=rng.choice([dtype, "e4m3"]), act_out=rng.random() < 0.7)


def _pad32(n):
    return (n + 31) // 32 * 32


def _scale_shape(fmt, rows, cols):
    """(tile rows, tiles along a row): each tile is 512 bytes."""
    return (rows + 127) // 128, (cols // _BLOCK[fmt] + 3) // 4


def _packed_bytes(fmt, rows, cols):
    return rows * cols // (1 if fmt == "mxfp8" else 2) + rows * cols // _BLOCK[fmt]


def work(case):
    if case["op"] == "quantize":
        m, n = case["rows"], case["cols"]
        es, packed = _ES[case["dtype"]], _packed_bytes(case["fmt"], m, n)
        b = m * n * es + 2 * packed + m * n * 2
        if case["both"]:
            mp = _pad32(m)
            b += 2 * _packed_bytes(case["fmt"], n, mp) + n * mp * 2
        return {"bytes": b, "flops": 0}
    if case["op"] == "dense_fwd":
        m, k, n = case["M"], case["K"], case["N"]
        return {"bytes": m * k * 2 + _packed_bytes(case["fmt"], n, k) + m * n * 2 + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if case["op"] == "dense_bwd":
        m, k, n = case["M"], case["K"], case["N"]
        return {"bytes": m * n * 2 + _packed_bytes(case["fmt"], k, n) + _packed_bytes(case["fmt"], k, _pad32(m))
                + m * k * 2 + k * n * 2 + n * 4, "flops": 4 * m * n * k}
    m, f, es = case["M"], case["F"], _ES[case["dtype"]]
    n_in = 2 * f if case["act"] in _GATED else f
    dxs = 1 if case["dx"] == "e4m3" else es
    return {"bytes": m * f * es + _packed_bytes("mxfp8", m, n_in) + m * n_in * dxs + 4 * n_in
            + (m * f * es if case["act_out"] else 0), "flops": 0}


# --------------------------------------------------------------------- plain forms: packing ---


def _tile_scales(s, fmt):
    """[rows, blocks] scale bytes -> the tiled buffer."""
    rows, nb = s.shape
    rt, g = (rows + 127) // 128, (nb + 3) // 4
    p = torch.zeros(rt * 128, g * 4, dtype=torch.uint8, device=s.device)
    p[:rows, :nb] = s
    return p.view(rt, 4, 32, g, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(t, fmt, rows, cols):
    rt, g = _scale_shape(fmt, rows, cols)
    s = t.view(rt, g, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, g * 4)
    return s[:rows, : cols // _BLOCK[fmt]]


def _pow2(k):
    """2^k in fp32 for whole k from -127 to 127, exactly (2^-127 is subnormal)."""
    k = k.to(torch.int32)
    return torch.where(k == -127, torch.full_like(k, 0x400000), (k + 127) << 23).view(torch.float32)


def _e2m1_codes(v):
    """E2M1 codes of fp32 values: the nearest, ties to the even code, saturating."""
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0)).to(torch.uint8)
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _tensor_scale(amax):
    """fp32 scale of an NVFP4 tensor from its amax: 6 * 448 / amax."""
    s = torch.full_like(amax, 2688.0) / amax
    s = torch.where(torch.isinf(s) & (amax > 0), torch.full_like(s, _FLT_MAX), s)
    return torch.where((amax > 0) & torch.isfinite(amax), s, torch.ones_like(s))


def _pack(x, fmt, s=None):
    """[rows, cols] -> (codes, scale bytes [rows, blocks]); s: the fp32 tensor scale of NVFP4."""
    x = x.float()
    rows, cols = x.shape
    blk = _BLOCK[fmt]
    b = x.reshape(rows, cols // blk, blk)
    amax = b.abs().amax(-1)
    fine = torch.isfinite(amax)
    if fmt == "nvfp4":
        t = (amax * s) / torch.tensor(6.0, device=x.device)
        sb = torch.where(fine, t, torch.zeros_like(t)).clamp(max=448.0).to(torch.float8_e4m3fn)
        sf = sb.float()
        e = torch.where(sf > 0, s / sf, torch.zeros_like(sf))
        codes8 = sb.view(torch.uint8)
        scale = torch.where(fine, codes8, torch.full_like(codes8, 0x7F))
        v = b * e.unsqueeze(-1)
    else:
        bits = amax.contiguous().view(torch.int32)
        top_exp, top_mant = (2, 0x400000) if fmt == "mxfp4" else (8, 0x600000)
        c = (bits >> 23) - top_exp + ((bits & 0x7FFFFF) > top_mant).int()
        c = c.clamp(0, 254)
        scale = torch.where(fine, c, torch.full_like(c, 255)).to(torch.uint8)
        v = b * _pow2(127 - c).unsqueeze(-1)
    v = torch.where(fine.unsqueeze(-1), v, torch.zeros_like(v)).reshape(rows, cols)
    if fmt == "mxfp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale
    q = _e2m1_codes(v)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale


def _unpack(codes, scale, fmt, s_inv=None):
    """fp32 values of codes and [rows, blocks] scale bytes."""
    dev = codes.device
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(_E2M1 + tuple(-t for t in _E2M1), device=dev)
        q = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1)
        v = table[q.int()]
    rows, cols = v.shape
    blk = _BLOCK[fmt]
    if fmt == "nvfp4":
        f = scale.contiguous().view(torch.float8_e4m3fn).float()
    else:
        f = _pow2(scale.int() - 127)
        f = torch.where(scale == 255, torch.full_like(f, float("nan")), f)
    v = (v.reshape(rows, cols // blk, blk) * f.unsqueeze(-1)).reshape(rows, cols)
    return v if s_inv is None else v * s_inv


def _pad_t(x):
    """x^T with its rows (x's columns) filled up to whole blocks of 32 with zeros."""
    m, n = x.shape
    t = torch.zeros(n, _pad32(m), dtype=x.dtype, device=x.device)
    t[:, :m] = x.t()
    return t


# ------------------------------------------------------------------ plain forms: activation ---

_GELU_K0, _GELU_K1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(name, h):
    """(value, derivative) of relu, gelu (tanh form) or silu."""
    if name == "relu":
        return torch.where(h > 0, h, torch.zeros_like(h)), (h > 0).to(h.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-h))
        return h * s, s * (1.0 + h * (1.0 - s))
    u = _GELU_K0 * (h + _GELU_K1 * h * h * h)
    t = torch.tanh(u)
    return 0.5 * h * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * h * (1.0 - t * t) * _GELU_K0 * (1.0 + 3.0 * _GELU_K1 * h * h)


def _base(act):
    return {"swiglu": "silu", "geglu": "gelu", "reglu": "relu"}.get(act, act)


# ------------------------------------------------------------------------------------ state ---


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(*shape, generator=g, device=g.device) * std).to(dtype)


def _tokens(g, m, n, dtype, std=1.0):
    """Rows of normal values, one in a hundred eight times larger."""
    x = torch.randn(m, n, generator=g, device=g.device) * std
    x[0::100] *= 8.0
    return x.to(dtype)


def _scalars(dev, scale=1.0):
    """scale, scale_inv and amax of a quantizer: one-element fp32 tensors."""
    s = torch.tensor([scale], dtype=torch.float32, device=dev)
    return {"scale": s, "scale_inv": 1.0 / s, "amax": torch.zeros(1, dtype=torch.float32, device=dev)}


def _u8(dev, *shape):
    return torch.empty(*shape, dtype=torch.uint8, device=dev)


def _scale_buffer(dev, fmt, rows, cols):
    rt, g = _scale_shape(fmt, rows, cols)
    return _u8(dev, rt * g * 512)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    st = dict(case)
    if case["op"] == "quantize":
        m, n, fmt = case["rows"], case["cols"], case["fmt"]
        dt = _DT[case["dtype"]]
        weights = case["dtype"] == "f32"
        st["x"] = _normal(g, (m, n), 0.02, dt) if weights else _tokens(g, m, n, dt)
        st["q"] = _scalars(dev, 2688.0 / (0.2 if weights else 40.0))
        st["codes"] = _u8(dev, m, n if fmt == "mxfp8" else n // 2)
        st["scales"] = _scale_buffer(dev, fmt, m, n)
        st["out"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
        if case["both"]:
            mp = _pad32(m)
            st["codes_t"] = _u8(dev, n, mp // 2)
            st["scales_t"] = _scale_buffer(dev, fmt, n, mp)
            st["out_t"] = torch.empty(n, mp, dtype=torch.bfloat16, device=dev)
        return st
    if case["op"] in ("dense_fwd", "dense_bwd"):
        m, k, n, fmt = case["M"], case["K"], case["N"], case["fmt"]
        st["q"] = _scalars(dev, 2688.0 / 40.0)  # of the tensor that the call quantizes
        nv = fmt == "nvfp4"
        if case["op"] == "dense_fwd":
            # the weights, packed once: a row for each output
            w = _normal(g, (n, k), 0.02, torch.float32)
            s = _tensor_scale(w.abs().amax())
            st["w"], sc = _pack(w, fmt, s)
            st["w_scales"] = _tile_scales(sc, fmt)
            st["w_scale_inv"] = (1.0 / s).reshape(1) if nv else None
            st["x"] = _tokens(g, m, k, torch.bfloat16)
            st["b"] = _normal(g, (n,), 0.02, torch.bfloat16) if case["bias"] else None
            st["out"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
            return st
        # what the forward pass left: the weights with a row for each input, x^T
        w = _normal(g, (k, n), 0.02, torch.float32)
        s = _tensor_scale(w.abs().amax())
        st["w"], sc = _pack(w, fmt, s)
        st["w_scales"] = _tile_scales(sc, fmt)
        st["w_scale_inv"] = (1.0 / s).reshape(1) if nv else None
        x = _pad_t(_tokens(g, m, k, torch.bfloat16))
        s = _tensor_scale(x.float().abs().amax())
        st["xt"], sc = _pack(x, fmt, s)
        st["xt_scales"] = _tile_scales(sc, fmt)
        st["x_scale_inv"] = (1.0 / s).reshape(1) if nv else None
        st["dy"] = _tokens(g, m, n, torch.bfloat16)
        st["dx"] = torch.empty(m, k, dtype=torch.bfloat16, device=dev)
        st["dw"] = torch.empty(k, n, dtype=torch.bfloat16, device=dev)
        st["dbias"] = torch.empty(n, dtype=torch.float32, device=dev)
        return st
    m, f = case["M"], case["F"]
    dt = _DT[case["dtype"]]
    n_in = 2 * f if case["act"] in _GATED else f
    st["codes"], sc = _pack(_tokens(g, m, n_in, dt), "mxfp8")
    st["scales"] = _tile_scales(sc, "mxfp8")
    st["dy"] = _normal(g, (m, f), 1.0, dt)
    st["q"] = _scalars(dev, 32.0)
    st["dx_buf"] = torch.empty(m, n_in, dtype=torch.uint8 if case["dx"] == "e4m3" else _DT[case["dx"]], device=dev)
    st["dbias"] = torch.empty(n_in, dtype=torch.float32, device=dev)
    st["a"] = torch.empty(m, f, dtype=dt, device=dev) if case["act_out"] else None
    return st


# -------------------------------------------------------------------------------------- run ---


def run(st):
    return (_run_own if own else _run_plain)(st)


def _quantizer(te, st, mode):
    """The amax is asked for where this call's scale comes from it, or the pass returns it."""
    q = st["q"]
    amax = q["amax"] if mode == "current" or st["op"] == "ckpt_bwd" else None
    return te.Quantizer.from_tensors(q["scale"], q["scale_inv"], amax, mode=mode)


def _run_own(st):
    import fp8_transformer_gb300 as te
    op = st["op"]
    if op == "quantize":
        fmt = st["fmt"]
        q = _quantizer(te, st, st["scaling"]) if fmt == "nvfp4" else None
        inv = st["q"]["scale_inv"] if fmt == "nvfp4" else None
        te.te_block_quantize(st["x"], fmt, codes=st["codes"], scales=st["scales"], codes_t=st.get("codes_t"),
                             scales_t=st.get("scales_t"), q=q)
        te.te_block_dequantize(st["codes"], st["scales"], fmt, st["out"], scale_inv=inv)
        if not st["both"]:
            return {"values": st["out"]}
        te.te_block_dequantize(st["codes_t"], st["scales_t"], fmt, st["out_t"], scale_inv=inv)
        return {"values": st["out"], "values_t": st["out_t"]}
    if op == "dense_fwd":
        q = _quantizer(te, st, st["scaling"]) if st["fmt"] == "nvfp4" else None
        te.te_dense_fp4_fwd(st["x"], st["w"], st["w_scales"], st["out"], st["fmt"], bias=st["b"], q=q,
                            kernel_scale_inv=st["w_scale_inv"])
        return {"out": st["out"]}
    if op == "dense_bwd":
        q = _quantizer(te, st, st["scaling"]) if st["fmt"] == "nvfp4" else None
        te.te_dense_fp4_bwd(st["dy"], st["w"], st["w_scales"], st["xt"], st["xt_scales"], st["dx"], st["dw"],
                            st["fmt"], dbias=st["dbias"], q=q, kernel_scale_inv=st["w_scale_inv"],
                            x_scale_inv=st["x_scale_inv"])
        return {"dx": st["dx"], "dw": st["dw"], "dbias": st["dbias"]}
    q = _quantizer(te, st, "delayed") if st["dx"] == "e4m3" else None
    te.te_dact_dbias_ckpt(st["dy"], st["codes"], st["scales"], st["act"], st["dx_buf"], dbias=st["dbias"],
                          act_out=st["a"], q=q)
    return _ckpt_outputs(st, st["dx_buf"], st["dbias"], st["a"], st["q"]["amax"])


def _ckpt_outputs(st, dx, dbias, a, amax):
    r = {"dx": dx.view(torch.float8_e4m3fn) if st["dx"] == "e4m3" else dx, "dbias": dbias}
    if st["act_out"]:
        r["act"] = a
    if st["dx"] == "e4m3":
        r["amax"] = amax
    return r


def _plain_scale(st, x):
    if st["fmt"] != "nvfp4":
        return None
    return _tensor_scale(x.float().abs().amax()) if st["scaling"] == "current" else st["q"]["scale"]


def _round_trip(x, fmt, s):
    codes, sc = _pack(x, fmt, s)
    return _unpack(codes, sc, fmt, None if s is None else 1.0 / s)


def _run_plain(st):
    op = st["op"]
    if op == "quantize":
        x, fmt = st["x"], st["fmt"]
        s = _plain_scale(st, x)
        r = {"values": _round_trip(x, fmt, s).to(torch.bfloat16)}
        if st["both"]:
            r["values_t"] = _round_trip(_pad_t(x), fmt, s).to(torch.bfloat16)
        return r
    if op == "dense_fwd":
        fmt, (n, k2) = st["fmt"], st["w"].shape
        x = _round_trip(st["x"], fmt, _plain_scale(st, st["x"]))
        w = _unpack(st["w"], _untile_scales(st["w_scales"], fmt, n, 2 * k2), fmt, st["w_scale_inv"])
        out = x @ w.t()
        if st["b"] is not None:
            out = out + st["b"].float()
        return {"out": out.to(torch.bfloat16)}
    if op == "dense_bwd":
        fmt, (k, n2) = st["fmt"], st["w"].shape
        s = _plain_scale(st, st["dy"])
        w = _unpack(st["w"], _untile_scales(st["w_scales"], fmt, k, 2 * n2), fmt, st["w_scale_inv"])
        xt = _unpack(st["xt"], _untile_scales(st["xt_scales"], fmt, k, 2 * st["xt"].shape[1]), fmt, st["x_scale_inv"])
        dx = _round_trip(st["dy"], fmt, s) @ w.t()
        dw = xt @ _round_trip(_pad_t(st["dy"]), fmt, s).t()
        return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16),
                "dbias": st["dy"].double().sum(0).float()}
    f = st["F"]
    h = _unpack(st["codes"], _untile_scales(st["scales"], "mxfp8", *st["codes"].shape), "mxfp8")
    dy = st["dy"].float()
    if st["act"] in _GATED:
        a, d = _act(_base(st["act"]), h[:, :f])
        lin = h[:, f:]
        dx = torch.cat((dy * lin * d, dy * a), dim=1)
        a = a * lin
    else:
        a, d = _act(st["act"], h)
        dx = dy * d
    dbias, amax = dx.double().sum(0).float(), dx.abs().amax().reshape(1)
    if st["dx"] == "e4m3":
        dx = (dx * st["q"]["scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    else:
        dx = dx.to(_DT[st["dx"]])
    return _ckpt_outputs(st, dx, dbias, a.to(_DT[st["dtype"]]), amax)


# ------------------------------------------------------------------------------------ exact ---
# From the definitions, in 64 bits.  Where a format's definition rounds to 32 bits on the way (the
# tensor scale's products), so does this.


def _x_pow2(k):
    """2^k in fp64 for whole k, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _x_e4m3(v):
    """fp64 values rounded to E4M3 (nearest even, saturating), as fp64."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -6))
    step = _x_pow2(e - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _x_e2m1(v):
    """fp64 values rounded to E2M1 (nearest even, saturating), as fp64."""
    _, e = torch.frexp(v.abs().clamp(min=1.0, max=6.0))
    step = _x_pow2(e - 2)
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _x_round_trip(x, fmt, s=None):
    """The values that a [rows, cols] tensor's codes stand for, in fp64; s: the fp32 tensor scale."""
    rows, cols = x.shape
    b = x.double().reshape(rows, -1, _BLOCK[fmt])
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        s = s.double()
        sb = _x_e4m3(((amax * s).float().double() / 6.0).float().double())
        e = torch.where(sb > 0, (s / sb).float().double(), torch.zeros_like(sb))
        q = _x_e2m1((b * e).float().double())
        inv = (1.0 / s).float().double()
        return ((q * sb) * inv).reshape(rows, cols)
    m, e = torch.frexp(amax / _TOP[fmt])  # the smallest power of two at or above amax / top
    p = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    c = _x_pow2(p)
    q = _x_e4m3(b / c) if fmt == "mxfp8" else _x_e2m1(b / c)
    return (q * c).reshape(rows, cols)


def _x_read(codes, scales, fmt, s_inv):
    """The values of packed codes with tiled scales, in fp64."""
    rows, width = codes.shape
    dev = codes.device
    cols = width if fmt == "mxfp8" else 2 * width
    r = torch.arange(rows, device=dev).unsqueeze(1)
    b = torch.arange(cols // _BLOCK[fmt], device=dev).unsqueeze(0)
    tiles = (cols // _BLOCK[fmt] + 3) // 4
    byte = scales[((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4].double()

    def small(c, bits):  # a sign, an exponent and a mantissa of `bits` bits; 3 for E4M3, 1 for E2M1
        c = c.long()
        top = 4 if bits == 3 else 2
        mant, ex = c & ((1 << bits) - 1), (c >> bits) & ((1 << top) - 1)
        bias = 7 if bits == 3 else 1
        v = torch.where(ex > 0, (1 + mant.double() / (1 << bits)) * _x_pow2(ex - bias),
                        mant.double() / (1 << bits) * 2.0 ** (1 - bias))
        return torch.where((c >> (bits + top)) & 1 == 1, -v, v)

    if fmt == "mxfp8":
        v = small(codes, 3)
    else:
        v = torch.empty(rows, cols, dtype=torch.float64, device=dev)
        v[:, 0::2], v[:, 1::2] = small(codes % 16, 1), small(codes // 16, 1)
    f = small(byte.long(), 3) if fmt == "nvfp4" else _x_pow2(byte - 127)
    v = (v.reshape(rows, -1, _BLOCK[fmt]) * f.unsqueeze(-1)).reshape(rows, cols)
    return v if s_inv is None else v * s_inv.double()


def _x_scale(st, x):
    if st["fmt"] != "nvfp4":
        return None
    return (torch.tensor(2688.0, dtype=torch.float64, device=x.device) / x.double().abs().amax()).float() if st["scaling"] == "current" else st["q"]["scale"]


def exact(case, seed):
    if "M" in case and "K" in case and case["M"] * case["K"] * case["N"] > 2e12:
        return None  # over 20 seconds in 64 bits
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        s = _x_scale(st, st["x"])
        r = {"values": _x_round_trip(st["x"], case["fmt"], s)}
        if case["both"]:
            m, n = st["x"].shape
            t = torch.nn.functional.pad(st["x"], (0, 0, 0, _pad32(m) - m)).t()
            r["values_t"] = _x_round_trip(t, case["fmt"], s)
        return r
    if op == "dense_fwd":
        x = _x_round_trip(st["x"], case["fmt"], _x_scale(st, st["x"]))
        out = x @ _x_read(st["w"], st["w_scales"], case["fmt"], st["w_scale_inv"]).t()
        return {"out": out if st["b"] is None else out + st["b"].double()}
    if op == "dense_bwd":
        s = _x_scale(st, st["dy"])
        m = case["M"]
        w = _x_read(st["w"], st["w_scales"], case["fmt"], st["w_scale_inv"])
        xt = _x_read(st["xt"], st["xt_scales"], case["fmt"], st["x_scale_inv"])
        dyt = torch.nn.functional.pad(st["dy"], (0, 0, 0, _pad32(m) - m)).t()
        return {"dx": _x_round_trip(st["dy"], case["fmt"], s) @ w.t(),
                "dw": xt @ _x_round_trip(dyt, case["fmt"], s).t(), "dbias": st["dy"].double().sum(0)}
    f, act = case["F"], case["act"]
    h = _x_read(st["codes"], st["scales"], "mxfp8", None)
    dy = st["dy"].double()
    gate = h[:, :f]
    if _base(act) == "relu":
        a, d = gate.clamp(min=0), (gate > 0).double()
    elif _base(act) == "silu":
        sg = torch.sigmoid(gate)
        a, d = gate * sg, sg + gate * sg * torch.sigmoid(-gate)
    else:
        k0 = math.sqrt(2 / math.pi)
        th = torch.tanh(k0 * (gate + 0.044715 * gate ** 3))
        a = gate * (1 + th) / 2
        d = (1 + th) / 2 + gate / 2 * (1 - th ** 2) * k0 * (1 + 3 * 0.044715 * gate ** 2)
    if act in _GATED:
        dx = torch.cat((dy * h[:, f:] * d, dy * a), dim=1)
        a = a * h[:, f:]
    else:
        dx = dy * d
    r = {"dx": dx, "dbias": dx.sum(0)}
    if case["dx"] == "e4m3":
        r["dx"], r["amax"] = _x_e4m3(dx * st["q"]["scale"].double()), dx.abs().amax().reshape(1)
    if case["act_out"]:
        r["act"] = a
    return r

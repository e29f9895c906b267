"""What is measured of the operators that tie the block into a layer: the norms around a residual
stream, the product that ends in it, and the norm and clipping of the gradients that are left.

  residual norm   p = norm(y) or y;  x_out = a r + gate p;  out = norm(x_out)
  dense residual  out = a r + gate act(x W + b)
  clipping        n = sqrt(sum of all g^2);  out = g min(1, max_norm / (n + eps))

A gate is [H] or [G, H]: each of its rows serves M / G neighbouring tokens (one sequence's).
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4, "e4m3": 1}
_EPS = 1e-6


# ------------------------------------------------------------------------------- the cases ---


def listed():
    return [
        # one token that generates: the block's output joins the stream, the next block's norm
        dict(name="norm one token", op="norm_fwd", norm="rmsnorm", M=1, H=4096, dtype="bf16", res="bf16",
             out="bf16", post=False, gate=0, scale=1.0),
        # a training batch, LayerNorm, a learned scale for each channel of the block's output
        dict(name="norm training", op="norm_fwd", norm="layernorm", M=16384, H=4096, dtype="bf16", res="bf16",
             out="bf16", post=False, gate=1, scale=1.0),
        # prompts of eight sequences with a gate each, norms on both sides of the block, an fp32
        # stream, the next product in FP8
        dict(name="norm prompts fp8", op="norm_fwd", norm="rmsnorm", M=1000, H=8192, dtype="bf16", res="f32",
             out="e4m3", post=True, gate=8, scale=1.0),
        # the gradient of a layer with norms on both sides of the block, at full size
        dict(name="norm backward both sides", op="norm_bwd", norm="rmsnorm", M=8192, H=4096, dtype="bf16",
             res="bf16", out="bf16", post=True, gate=0, scale=1.0),
        # three short sequences with gates, LayerNorm on both sides, fp32 stream, scaled residual
        dict(name="norm backward gated", op="norm_bwd", norm="layernorm", M=777, H=2048, dtype="bf16",
             res="f32", out="bf16", post=True, gate=3, scale=0.5),
        # one token through the down projection into the stream
        dict(name="dense one token", op="dense_fwd", M=1, K=14336, N=4096, fp8=False, act="identity",
             bias=False, gate=0, scale=1.0),
        # an odd number of sequences that generate, FP8
        dict(name="dense 17 tokens fp8", op="dense_fwd", M=17, K=16384, N=4096, fp8=True, act="identity",
             bias=True, gate=1, scale=1.0),
        # a prompt through a square layer with its activation
        dict(name="dense prompt", op="dense_fwd", M=1000, K=8192, N=8192, fp8=False, act="gelu", bias=True,
             gate=4, scale=1.0),
        # a training batch through the down projection
        dict(name="dense training", op="dense_fwd", M=8192, K=14336, N=4096, fp8=False, act="identity",
             bias=False, gate=0, scale=1.0),
        # the gradient of a layer with its activation and gate, ragged token count
        dict(name="dense backward", op="dense_bwd", M=4100, K=4096, N=4096, fp8=False, act="gelu", bias=True,
             gate=1, scale=1.0),
        # the vectors of a deep model: many small gradients, cut out of one buffer
        dict(name="clip many small", op="clip", count=290, lo=16, hi=16384, dtype="mixed", sizes=7, big=0,
             max_norm=1.0),
        # one gated block's gradients: two weights in one bucket, the vectors in another
        dict(name="clip block", op="clip", count=1, lo=40960, hi=40960, dtype="f32", sizes=1,
             big=4096 * 3 * 14336, max_norm=1.0),
    ]


def _size(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd", "dense_fwd", "dense_fwd", "dense_bwd", "clip"])
    if op in ("norm_fwd", "norm_bwd"):
        gate = rng.choice([0, 1, rng.randint(2, 9)])
        M, H = _size(rng, 1, 12000), _size(rng, 64, 8192, 8)
        if M * H > 1 << 26:
            M = (1 << 26) // H
        M = max(1, M // max(gate, 1)) * max(gate, 1)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, norm=rng.choice(["layernorm", "rmsnorm"]), M=M, H=H, dtype=dtype,
                    res="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                    out=rng.choice([dtype, "e4m3"]) if op == "norm_fwd" else dtype,
                    post=rng.random() < 0.5, gate=gate, scale=rng.choice([1.0, 0.5]))
    if op in ("dense_fwd", "dense_bwd"):
        gate = rng.choice([0, 0, 1, rng.randint(2, 5)])
        M, K, N = _size(rng, 1, 6000), _size(rng, 64, 14336, 16), _size(rng, 64, 8192, 16)
        M = min(M, int(2e11) // (K * N) + 1)
        M = max(1, M // max(gate, 1)) * max(gate, 1)
        return dict(op=op, M=M, K=K, N=N, fp8=rng.random() < 0.4,
                    act=rng.choice(["identity", "identity", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                    gate=gate, scale=rng.choice([1.0, 0.5]))
    return dict(op=op, count=_size(rng, 1, 400), lo=1, hi=_size(rng, 100, 300000),
                dtype=rng.choice(["bf16", "f32", "mixed"]), sizes=rng.randint(1, 10 ** 6),
                big=rng.choice([0, _size(rng, 1 << 16, 1 << 25)]), max_norm=rng.choice([1.0, 1e9]))


def _sizes(case):
    """The element counts of a list of gradients, the large one first."""
    r = random.Random(case["sizes"])
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    n = [int(round(math.exp(r.uniform(lo, hi)))) for _ in range(case["count"])]
    return ([case["big"]] if case["big"] else []) + n


def _types(case):
    """Their types: the large one's is bf16."""
    n = len(_sizes(case))
    if case["dtype"] == "mixed":
        t = ["bf16" if i % 3 else "f32" for i in range(n)]
    else:
        t = [case["dtype"]] * n
    if case["big"]:
        t[0] = "bf16"
    return t


def work(case):
    op = case["op"]
    if op == "clip":
        return {"bytes": sum(2 * n * _ES[t] for n, t in zip(_sizes(case), _types(case))), "flops": 0}
    if op in ("norm_fwd", "norm_bwd"):
        m, h, e, r = case["M"], case["H"], _ES[case["dtype"]], _ES[case["res"]]
        vec = 2 * (2 if case["post"] else 1) + case["gate"]
        stats = 4 * m * (4 if case["post"] else 2)
        if op == "norm_fwd":
            return {"bytes": m * h * (e + 2 * r + _ES[case["out"]]) + vec * h * e + stats, "flops": 0}
        y = 2 * e if case["post"] or case["gate"] else e  # dy, and y where the gradient depends on it
        return {"bytes": m * h * (e + 3 * r + y) + vec * h * (e + 4) + stats, "flops": 0}
    m, k, n, e = case["M"], case["K"], case["N"], 1 if case["fp8"] else 2
    if op == "dense_fwd":
        return {"bytes": m * k * e + k * n * e + m * n * 4 + 2 * n * (case["gate"] + case["bias"]),
                "flops": 2 * m * n * k}
    z = 2 if case["gate"] or case["act"] != "identity" else 0
    return {"bytes": m * n * (4 + z) + 2 * (m * k + k * n) + (m * k + k * n) * e + 6 * n * (case["gate"] + case["bias"]),
            "flops": 4 * m * n * k}


# ------------------------------------------------------------------------------ plain forms ---

_GELU_K0, _GELU_K1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(name, z):
    """(value, derivative) of identity, relu, gelu (tanh form) or silu."""
    if name == "identity":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).to(z.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    t = torch.tanh(_GELU_K0 * (z + _GELU_K1 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _GELU_K0 * (1.0 + 3.0 * _GELU_K1 * z * z)


def _norm(x, gamma, beta, layernorm):
    """(norm of the rows, row means, reciprocal deviations) in fp32."""
    mu = x.mean(1) if layernorm else torch.zeros_like(x[:, 0])
    d = x - mu[:, None]
    rs = 1.0 / torch.sqrt((d * d).mean(1) + _EPS)
    out = d * rs[:, None] * gamma
    return (out + beta if layernorm else out), mu, rs


def _norm_grad(d, xhat, rs, layernorm):
    """Gradient of the norm's input from that of its normalized rows."""
    c = (d * xhat).mean(1, keepdim=True)
    g = d - xhat * c
    if layernorm:
        g = g - d.mean(1, keepdim=True)
    return g * rs[:, None]


def _rows(gate, m):
    """The gate of each row: [G, H] -> [M, H]."""
    return gate.float().repeat_interleave(m // gate.shape[0], 0)


def _column_sum(t, groups=1):
    """fp32 column sums of each group of rows, added in 64 bits: [groups, N]."""
    return t.reshape(groups, -1, t.shape[1]).double().sum(1).float()


def _e4m3(v):
    """fp32 values as E4M3, saturating."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


# ------------------------------------------------------------------------------------ state ---


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _normal(g, shape, std, dtype, mean=0.0):
    return (torch.randn(*shape, generator=g, device=g.device) * std + mean).to(dtype)


def _tokens(g, m, n, dtype, std=1.0):
    """Rows of normal values, one in a hundred eight times larger."""
    x = torch.randn(m, n, generator=g, device=g.device) * std
    x[0::100] *= 8.0
    return x.to(dtype)


def _quantizer_scalars(dev, scale):
    s = torch.tensor([scale], dtype=torch.float32, device=dev)
    return {"scale": s, "scale_inv": 1.0 / s, "amax": torch.zeros(1, dtype=torch.float32, device=dev)}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    st = dict(case)
    op = case["op"]
    if op == "clip":
        st["grads"], st["outs"] = [], []
        sizes, types = _sizes(case), _types(case)
        for name in ("bf16", "f32"):
            total = sum(n for n, t in zip(sizes, types) if t == name)
            st["flat_" + name] = (_normal(g, (total,), 0.01, _DT[name]) if total else None,
                                  torch.empty(total, dtype=_DT[name], device=dev))
        at = {"bf16": 0, "f32": 0}
        for n, t in zip(sizes, types):
            src, dst = st["flat_" + t]
            st["grads"].append(src[at[t]:at[t] + n])
            st["outs"].append(dst[at[t]:at[t] + n])
            at[t] += n
        st["norm"] = torch.empty(1, dtype=torch.float32, device=dev)
        if own:  # the list that a training program keeps beside its parameters
            import fp8_transformer_gb300 as te
            st["list"] = te.GradList(st["grads"], st["outs"])
        return st
    m = case["M"]
    if op in ("norm_fwd", "norm_bwd"):
        h, dt, rt = case["H"], _DT[case["dtype"]], _DT[case["res"]]
        ln = case["norm"] == "layernorm"
        st["gamma"] = _normal(g, (h,), 0.1, dt, 1.0)
        st["beta"] = _normal(g, (h,), 0.1, dt) if ln else None
        st["post_gamma"] = _normal(g, (h,), 0.1, dt, 1.0) if case["post"] else None
        st["post_beta"] = _normal(g, (h,), 0.1, dt) if ln and case["post"] else None
        st["gate"] = _normal(g, (case["gate"], h), 0.3, dt, 0.5) if case["gate"] else None
        st["y"] = _tokens(g, m, h, dt)
        st["residual"] = _tokens(g, m, h, rt, 2.0)
        stats = [torch.empty(m, dtype=torch.float32, device=dev) for _ in range(4)]
        st["mu"], st["rs"], st["post_mu"], st["post_rs"] = stats
        if op == "norm_fwd":
            st["x_out"] = torch.empty(m, h, dtype=rt, device=dev)
            st["out"] = torch.empty(m, h, dtype=torch.uint8 if case["out"] == "e4m3" else _DT[case["out"]], device=dev)
            st["q"] = _quantizer_scalars(dev, 32.0)
            return st
        # what the forward pass left, and the gradients that reach its two outputs
        fwd = _norm_fwd_plain(st)
        st["x_out"] = fwd["x_out"]
        for k in ("mu", "rs", "post_mu", "post_rs"):
            if fwd.get(k) is not None:
                st[k] = fwd[k]
        del st["residual"]
        st["dout"] = _normal(g, (m, h), 1.0, dt)
        st["dx_out"] = _normal(g, (m, h), 1.0, rt)
        st["dresidual"] = torch.empty(m, h, dtype=rt, device=dev)
        st["dy"] = torch.empty(m, h, dtype=dt, device=dev)
        vec = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)  # noqa: E731
        st["dgamma"], st["dbeta"] = vec(h), vec(h) if ln else None
        st["dpost_gamma"] = vec(h) if case["post"] else None
        st["dpost_beta"] = vec(h) if ln and case["post"] else None
        st["dgate"] = vec(case["gate"], h) if case["gate"] else None
        return st
    k, n, bf = case["K"], case["N"], torch.bfloat16
    x, w = _tokens(g, m, k, bf), _normal(g, (k, n), 0.02, bf)
    st["x_inv"] = st["w_inv"] = None
    if case["fp8"]:  # the quantizers' scales of earlier steps
        sx, sw = _quantizer_scalars(dev, 448.0 / 48.0), _quantizer_scalars(dev, 448.0 / 0.15)
        x, w = _e4m3(x.float() * sx["scale"]), _e4m3(w.float() * sw["scale"])
        st["x_inv"], st["w_inv"] = sx["scale_inv"], sw["scale_inv"]
    st["x"], st["w"] = x, w
    st["bias"] = _normal(g, (n,), 0.1, bf) if case["bias"] else None
    st["gate"] = _normal(g, (case["gate"], n), 0.3, bf, 0.5) if case["gate"] else None
    if op == "dense_fwd":
        st["residual"] = _tokens(g, m, n, bf, 2.0)
        st["out"] = torch.empty(m, n, dtype=bf, device=dev)
        return st
    st["z"] = _normal(g, (m, n), 1.5, bf)  # of the size that the forward pass stores
    st["dout"] = _normal(g, (m, n), 1.0, bf)
    st["q"] = _quantizer_scalars(dev, 448.0 / 24.0)
    st["dx"] = torch.empty(m, k, dtype=bf, device=dev)
    st["dw"] = torch.empty(k, n, dtype=bf, device=dev)
    st["dresidual"] = torch.empty(m, n, dtype=bf, device=dev) if case["scale"] != 1.0 else None
    st["dbias"] = torch.empty(n, dtype=torch.float32, device=dev) if case["bias"] else None
    st["dgate"] = torch.empty(case["gate"], n, dtype=torch.float32, device=dev) if case["gate"] else None
    return st


# -------------------------------------------------------------------------------------- run ---


def run(st):
    return (_run_own if own else _run_plain)(st)


def _some(**kw):
    return {k: v for k, v in kw.items() if v is not None}


def _run_own(st):
    import fp8_transformer_gb300 as te
    op = st["op"]
    if op == "clip":
        te.te_clip_grad_norm(st["list"], st["max_norm"], st["norm"], epsilon=_EPS)
        return _clip_outputs(st, st["norm"])
    if op == "norm_fwd":
        q = None
        if st["out"].dtype == torch.uint8:
            q = te.Quantizer.from_tensors(st["q"]["scale"], st["q"]["scale_inv"], st["q"]["amax"])
        post = dict(post_mu=st["post_mu"], post_rsigma=st["post_rs"]) if st["post"] else {}
        te.te_residual_norm_fwd(st["y"], st["residual"], st["gamma"], st["beta"], st["x_out"], st["out"],
                                norm_type=st["norm"], epsilon=_EPS, post_gamma=st["post_gamma"],
                                post_beta=st["post_beta"], gate=st["gate"], residual_scale=st["scale"], q=q,
                                mu=st["mu"], rsigma=st["rs"], **post)
        return _norm_fwd_outputs(st, st["x_out"], st["out"], st["q"]["amax"])
    if op == "norm_bwd":
        post = dict(post_mu=st["post_mu"], post_rsigma=st["post_rs"]) if st["post"] else {}
        te.te_residual_norm_bwd(st["dout"], st["dx_out"], st["x_out"], st["mu"], st["rs"], st["gamma"],
                                st["dresidual"], st["dy"], st["dgamma"], dbeta=st["dbeta"],
                                y=st["y"] if st["post"] or st["gate"] is not None else None,
                                post_gamma=st["post_gamma"], post_beta=st["post_beta"], gate=st["gate"],
                                residual_scale=st["scale"], dpost_gamma=st["dpost_gamma"],
                                dpost_beta=st["dpost_beta"], dgate=st["dgate"], norm_type=st["norm"], **post)
        return _some(**{k: st[k] for k in ("dresidual", "dy", "dgamma", "dbeta", "dpost_gamma", "dpost_beta", "dgate")})
    if op == "dense_fwd":
        te.te_dense_residual_fwd(st["x"], st["w"], st["residual"], st["out"], bias=st["bias"],
                                 activation=st["act"], gate=st["gate"], residual_scale=st["scale"],
                                 x_scale_inv=st["x_inv"], kernel_scale_inv=st["w_inv"])
        return {"out": st["out"]}
    q = te.Quantizer.from_tensors(st["q"]["scale"], st["q"]["scale_inv"], None) if st["fp8"] else None
    te.te_dense_residual_bwd(st["dout"], st["x"], st["w"], st["dx"], st["dw"], dresidual=st["dresidual"],
                             saved_z=st["z"] if st["act"] != "identity" or st["gate"] is not None else None,
                             activation=st["act"], gate=st["gate"], residual_scale=st["scale"], dbias=st["dbias"],
                             dgate=st["dgate"], q=q, x_scale_inv=st["x_inv"], kernel_scale_inv=st["w_inv"])
    return _some(**{k: st[k] for k in ("dx", "dw", "dresidual", "dbias", "dgate")})


def _clip_outputs(st, norm):
    """The norm, and the buffers that the clipped gradients are cut from."""
    return _some(norm=norm, **{t: st["flat_" + t][1] for t in ("bf16", "f32") if st["flat_" + t][0] is not None})


def _norm_fwd_outputs(st, x_out, out, amax):
    if out.dtype == torch.uint8:
        out = out.view(torch.float8_e4m3fn)
    r = {"x_out": x_out, "out": out}
    if out.dtype == torch.float8_e4m3fn:
        r["amax"] = amax
    return r


def _norm_fwd_plain(st):
    """Every result of the forward pass, the statistics among them."""
    ln, m = st["norm"] == "layernorm", st["M"]
    r = {}
    p = st["y"].float()
    if st["post"]:
        p, r["post_mu"], r["post_rs"] = _norm(p, st["post_gamma"].float(), st["post_beta"].float() if ln else None, ln)
    if st["gate"] is not None:
        p = p * _rows(st["gate"], m)
    x = st["scale"] * st["residual"].float() + p
    r["norm"], r["mu"], r["rs"] = _norm(x, st["gamma"].float(), st["beta"].float() if ln else None, ln)
    r["x_out"] = x.to(_DT[st["res"]])
    return r


def _run_plain(st):
    op = st["op"]
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device=st["grads"][0].device)
        for t in st["grads"]:
            total = total + (t.double() * t.double()).sum()
        n = torch.sqrt(total)
        c = torch.clamp(st["max_norm"] / (n + _EPS), max=1.0).float()
        for t, o in zip(st["grads"], st["outs"]):
            o.copy_(t.float() * c)
        return _clip_outputs(st, n.float().reshape(1))
    if op == "norm_fwd":
        r = _norm_fwd_plain(st)
        v = r["norm"]
        if st["out"].dtype == torch.uint8:
            out = _e4m3(v * st["q"]["scale"])
        else:
            out = v.to(st["out"].dtype)
        return _norm_fwd_outputs(st, r["x_out"], out, v.abs().amax().reshape(1))
    m = st["M"]
    if op == "norm_bwd":
        ln = st["norm"] == "layernorm"
        dout = st["dout"].float()
        xhat = (st["x_out"].float() - (st["mu"][:, None] if ln else 0.0)) * st["rs"][:, None]
        dx = st["dx_out"].float() + _norm_grad(dout * st["gamma"].float(), xhat, st["rs"], ln)
        r = {"dresidual": (st["scale"] * dx).to(_DT[st["res"]])}
        sums = {"dgamma": _column_sum(dout * xhat)[0], "dbeta": _column_sum(dout)[0] if ln else None}
        p = phat = st["y"].float()
        if st["post"]:
            phat = (p - (st["post_mu"][:, None] if ln else 0.0)) * st["post_rs"][:, None]
            p = phat * st["post_gamma"].float()
            if ln:
                p = p + st["post_beta"].float()
        dp = dx
        if st["gate"] is not None:
            dp = dx * _rows(st["gate"], m)
            sums["dgate"] = _column_sum(dx * p, st["gate"].shape[0])
        if st["post"]:
            sums["dpost_gamma"] = _column_sum(dp * phat)[0]
            sums["dpost_beta"] = _column_sum(dp)[0] if ln else None
            dp = _norm_grad(dp * st["post_gamma"].float(), phat, st["post_rs"], ln)
        r["dy"] = dp.to(_DT[st["dtype"]])
        return _some(**r, **sums)
    x, w = st["x"].float(), st["w"].float()
    if st["fp8"]:
        x, w = x * st["x_inv"], w * st["w_inv"]
    if op == "dense_fwd":
        z = x @ w
        if st["bias"] is not None:
            z = z + st["bias"].float()
        v = _act(st["act"], z)[0]
        if st["gate"] is not None:
            v = v * _rows(st["gate"], m)
        return {"out": (st["scale"] * st["residual"].float() + v).to(torch.bfloat16)}
    dout = st["dout"].float()
    r = {}
    a, d = _act(st["act"], st["z"].float())
    dz = dout * d
    if st["gate"] is not None:
        r["dgate"] = _column_sum(dout * a, st["gate"].shape[0])
        dz = dz * _rows(st["gate"], m)
    if st["bias"] is not None:
        r["dbias"] = _column_sum(dz)[0]
    if st["scale"] != 1.0:
        r["dresidual"] = (st["scale"] * dout).to(torch.bfloat16)
    # the operand of both products, in their type
    dz = _e4m3(dz * st["q"]["scale"]).float() * st["q"]["scale_inv"] if st["fp8"] else dz.to(torch.bfloat16).float()
    r["dx"], r["dw"] = (dz @ w.t()).to(torch.bfloat16), (x.t() @ dz).to(torch.bfloat16)
    return r


# ------------------------------------------------------------------------------------ exact ---
# From the definitions, in 64 bits.  A product's operand that is stored in fewer bits is rounded here too.


def _x_round(v, bits, lowest):
    """fp64 values rounded to `bits` bits of significand (nearest even), steps no finer than those of 2^lowest."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** lowest))
    step = torch.ldexp(torch.ones_like(v), e - bits)
    return torch.round(v / step) * step


def _x_e4m3(v):
    return _x_round(v, 4, -6).clamp(-448.0, 448.0)


def _x_gate(st):
    if st["gate"] is None:
        return 1.0
    g = st["gate"].double()
    return g[torch.arange(st["M"], device=g.device) // (st["M"] // g.shape[0])]


def _x_act(name, z):
    if name == "identity":
        return z, 1.0
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(2 * u)  # (1 + tanh u) / 2
    return z * s, s + 2 * z * s * torch.sigmoid(-2 * u) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def _x_by_group(st, t):
    return torch.stack([c.sum(0) for c in t.chunk(st["gate"].shape[0])])


def exact(case, seed):
    if "K" in case and case["M"] * case["K"] * case["N"] > 2e12:
        return None  # over 20 seconds in 64 bits
    st = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        n = sum(t.double().square().sum() for t in st["grads"]).sqrt()
        c = min(1.0, case["max_norm"] / (n.item() + _EPS))
        return _some(norm=n.reshape(1), **{t: st["flat_" + t][0].double() * c for t in ("bf16", "f32")
                                           if st["flat_" + t][0] is not None})
    if op == "norm_fwd":
        ln = case["norm"] == "layernorm"

        def norm(v, gamma, beta):
            if ln:
                v = v - v.mean(-1, keepdim=True)
            v = v / (v.square().mean(-1, keepdim=True) + _EPS).sqrt() * gamma.double()
            return v + beta.double() if ln else v

        p = st["y"].double()
        if case["post"]:
            p = norm(p, st["post_gamma"], st["post_beta"])
        x = case["scale"] * st["residual"].double() + _x_gate(st) * p
        v = norm(x, st["gamma"], st["beta"])
        if case["out"] != "e4m3":
            return {"x_out": x, "out": v}
        return {"x_out": x, "out": _x_e4m3(v * st["q"]["scale"].double()), "amax": v.abs().amax().reshape(1)}
    if op == "norm_bwd":
        ln = case["norm"] == "layernorm"

        def hat(v, mu, rs):
            return (v.double() - mu.double()[:, None] if ln else v.double()) * rs.double()[:, None]

        def back(d, xh, rs):  # less its parts along the row of ones (LayerNorm) and along xhat
            h = d.shape[1]
            out = d - xh * ((d * xh).sum(-1, keepdim=True) / h)
            return (out - d.sum(-1, keepdim=True) / h if ln else out) * rs.double()[:, None]

        dout, xh = st["dout"].double(), hat(st["x_out"], st["mu"], st["rs"])
        dx = st["dx_out"].double() + back(dout * st["gamma"].double(), xh, st["rs"])
        r = {"dresidual": case["scale"] * dx, "dgamma": (dout * xh).sum(0), "dbeta": dout.sum(0) if ln else None}
        dp = dx * _x_gate(st)
        p = st["y"].double()
        if case["post"]:
            ph = hat(p, st["post_mu"], st["post_rs"])
            r["dpost_gamma"], r["dpost_beta"] = (dp * ph).sum(0), dp.sum(0) if ln else None
            p = ph * st["post_gamma"].double() + (st["post_beta"].double() if ln else 0.0)
            r["dy"] = back(dp * st["post_gamma"].double(), ph, st["post_rs"])
        else:
            r["dy"] = dp
        if st["gate"] is not None:
            r["dgate"] = _x_by_group(st, dx * p)
        return _some(**{k: r.get(k) for k in ("dresidual", "dy", "dgamma", "dbeta", "dpost_gamma", "dpost_beta", "dgate")})
    x, w = st["x"].double(), st["w"].double()
    if case["fp8"]:
        x, w = x * st["x_inv"].double(), w * st["w_inv"].double()
    if op == "dense_fwd":
        z = x @ w
        if st["bias"] is not None:
            z = z + st["bias"].double()
        return {"out": case["scale"] * st["residual"].double() + _x_gate(st) * _x_act(case["act"], z)[0]}
    dout = st["dout"].double()
    a, d = _x_act(case["act"], st["z"].double())
    dz = dout * _x_gate(st) * d
    r = {"dbias": dz.sum(0) if st["bias"] is not None else None,
         "dresidual": case["scale"] * dout if case["scale"] != 1.0 else None,
         "dgate": _x_by_group(st, dout * a) if st["gate"] is not None else None}
    dz = _x_e4m3(dz * st["q"]["scale"].double()) * st["q"]["scale_inv"].double() if case["fp8"] else _x_round(dz, 8, -126)
    return _some(dx=dz @ w.t(), dw=x.t() @ dz, dresidual=r["dresidual"], dbias=r["dbias"], dgate=r["dgate"])

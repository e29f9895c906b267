"""The LN-MLP block with its pre-activation kept in 8 bits: forward, then backward from the checkpoint.

The forward is the plain one's in every output, and its checkpoint is the packing of the plain
one's saved_h, byte for byte.  The backward is held, step by step, to the oracle's backward at the
values that the checkpoint stands for (exact in bf16), by the rules of the plain backward's test.
"""

import numpy as np
import pytest
import torch

import fp8_transformer_gb300 as te
from oracle import block as ob
from oracle import block_scaled as bs
from parity import np64
from steps import check_mlp_bwd
from workloads import make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
GATED = ("swiglu", "geglu", "reglu")


def quantizers(mode):
    if mode is None:
        return None
    if mode == "current":
        return te.QuantizerSet(**{k: te.Quantizer(mode="current") for k in ("x", "kernel1", "act", "kernel2", "grad")})
    return te.QuantizerSet(x=te.Quantizer(32.0), kernel1=te.Quantizer(2048.0), act=te.Quantizer(16.0),
                           kernel2=te.Quantizer(2048.0), grad=te.Quantizer(64.0))


def inputs(name, act, M, H, F):
    inp = make_inputs(name, device=DEV, M=M, H=H, F=F)
    if act is not None:
        inp["act"] = act
    if "dy" not in inp:
        inp["dy"] = make_inputs("gpt_ln_mlp_bwd", device=DEV, M=M, H=H, F=16, seed=1)["dy"]
    return inp


def forward(inp, mode, ckpt):
    M, H, F = inp["M"], inp["H"], inp["F"]
    F1 = 2 * F if inp["act"] in GATED else F
    dt = inp["x"].dtype
    qs = quantizers(mode)
    r = dict(qs=qs, out=torch.empty(M, H, dtype=dt, device=DEV),
             ln=torch.empty(M, H, dtype=torch.uint8 if mode else dt, device=DEV),
             mu=torch.empty(M, device=DEV), rs=torch.empty(M, device=DEV),
             act=torch.empty(M, F, dtype=torch.uint8 if mode else dt, device=DEV))
    kw = dict(norm_type=inp["norm"], zero_centered_gamma=inp["zero_centered_gamma"], activation_type=inp["act"],
              quantizer_set=qs, epsilon=inp["eps"], saved_ln_out=r["ln"], mu=r["mu"], rsigma=r["rs"],
              saved_act=r["act"])
    args = (inp["x"], inp["gamma"], inp["beta"], inp["w1"], inp["w2"], inp.get("b1"), inp.get("b2"), r["out"])
    if ckpt:
        n = te.block_scale_bytes("mxfp8", M, F1)
        codes = torch.full((M * F1 + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        scales = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        r["codes"], r["scales"] = codes[:M * F1].view(M, F1), scales[:n]
        te.te_layernorm_mlp_fwd_ckpt(*args, r["codes"], r["scales"], **kw)
        assert (codes[M * F1:] == 0xA5).all() and (scales[n:] == 0xA5).all()
    else:
        r["h"] = torch.empty(M, F1, dtype=dt, device=DEV)
        te.te_layernorm_mlp_fwd(*args, saved_h=r["h"], **kw)
    torch.cuda.synchronize()
    assert te.get_device_status() == 0
    return r


@pytest.mark.parametrize("name,act,M,H,F", [("gpt_ln_mlp_bwd", None, 300, 512, 800),
                                            ("gpt_ln_mlp_bwd", "relu", 1, 256, 32),
                                            ("llama_rms_mlp", None, 256, 512, 544),
                                            ("llama_rms_mlp", "geglu", 77, 256, 96),
                                            ("tiny_ln_mlp", None, 64, 128, 512)])
@pytest.mark.parametrize("mode", [None, "delayed", "current"])
def test_forward_is_the_plain_one_with_its_preactivation_packed(name, act, M, H, F, mode):
    inp = inputs(name, act, M, H, F)
    if inp["x"].dtype == torch.float32:
        inp["dy"] = None
    a, b = forward(inp, mode, False), forward(inp, mode, True)
    for k in ("out", "ln", "mu", "rs", "act"):
        assert torch.equal(a[k], b[k]), k
    c, s = bs.pack(np64(a["h"]), "mxfp8")
    assert np.array_equal(b["codes"].cpu().numpy(), c)
    assert np.array_equal(b["scales"].cpu().numpy(), bs.tile_scales(s))


def backward(inp, f, **over):
    M, H, F = inp["M"], inp["H"], inp["F"]
    gated = inp["act"] in GATED
    F1 = 2 * F if gated else F
    dt = torch.bfloat16
    g = dict(f, dx=torch.empty(M, H, dtype=dt, device=DEV), dgamma=torch.empty(H, device=DEV),
             dbeta=torch.empty(H, device=DEV), dw1=torch.empty(H, F1, dtype=dt, device=DEV),
             dw2=torch.empty(F, H, dtype=dt, device=DEV), db1=torch.empty(F1, device=DEV),
             db2=torch.empty(H, device=DEV),
             dh=torch.empty(M, F1, dtype=torch.uint8 if f["qs"] else dt, device=DEV))
    te.te_layernorm_mlp_bwd_ckpt(inp["dy"], inp["x"], inp["gamma"], inp["w1"], inp["w2"], f["codes"], f["scales"],
                                 f["ln"], f["mu"], f["rs"], g["dx"], g["dgamma"], g["dw1"], g["dw2"],
                                 dbeta=g["dbeta"], dbias1=g["db1"], dbias2=g["db2"], norm_type=inp["norm"],
                                 zero_centered_gamma=inp["zero_centered_gamma"], activation_type=inp["act"],
                                 quantizer_set=f["qs"], saved_dh=g["dh"], **over)
    return g


@pytest.mark.parametrize("name,act,M,H,F", [("gpt_ln_mlp_bwd", None, 300, 512, 800),
                                            ("gpt_ln_mlp_bwd", "silu", 33, 256, 160),
                                            ("llama_rms_mlp", None, 256, 512, 544),
                                            ("llama_rms_mlp", "reglu", 130, 256, 96)])
@pytest.mark.parametrize("mode", [None, "delayed", "current"])
def test_backward_from_the_checkpoint(name, act, M, H, F, mode):
    inp = inputs(name, act, M, H, F)
    f = forward(inp, mode, True)
    g = backward(inp, f)
    torch.cuda.synchronize()
    assert te.get_device_status() == 0
    # the values that the checkpoint stands for: 4 significant bits, exact in bf16
    g["h"] = te.te_block_dequantize(f["codes"], f["scales"], "mxfp8", torch.empty_like(f["codes"], dtype=torch.bfloat16))
    if inp["norm"] != "layernorm":
        assert int(g["dbeta"].count_nonzero().item()) == 0
        g["dbeta"] = None
    check_mlp_bwd(inp, g, mode is not None)


@pytest.mark.parametrize("act", ["gelu", "relu", "geglu", "swiglu"])
@pytest.mark.parametrize("mode", [None, "delayed"])
def test_an_overflow_before_the_activation_is_not_hidden(act, mode):
    """An infinite bias of one column: the gradients of its block's 32 columns are NaN, the others finite."""
    M, H, F = 70, 128, 96
    inp = inputs("gpt_ln_mlp_bwd" if act in ("gelu", "relu") else "llama_rms_mlp", act, M, H, F)
    F1 = 2 * F if act in GATED else F
    b1 = torch.zeros(F1, dtype=torch.bfloat16, device=DEV)
    b1[37] = float("inf")
    inp["b1"] = b1
    f = forward(inp, mode, True)
    g = backward(inp, f)
    torch.cuda.synchronize()
    of_act = torch.zeros(F, dtype=torch.bool, device=DEV)
    of_act[32:64] = True
    of_h = torch.cat([of_act, of_act]) if act in GATED else of_act
    assert torch.equal(torch.isnan(g["db1"]), of_h)
    assert torch.isnan(g["dw1"][:, of_h]).all() and torch.isnan(g["dw2"][of_act]).all()
    assert torch.isfinite(g["dw1"][:, ~of_h]).all() and torch.isfinite(g["dw2"][~of_act]).all()
    assert torch.isfinite(g["db1"][~of_h]).all()


def test_backward_is_the_same_on_every_run_and_in_a_graph():
    inp = inputs("llama_rms_mlp", None, 200, 256, 288)
    f = forward(inp, None, True)
    ref = backward(inp, f)
    ws = torch.empty(te.workspace_size(te.binding.TE_OP_LAYERNORM_MLP_BWD, 200, 256, 288, te.binding.TE_BF16, False,
                                       te.binding.TE_BF16, te.binding.TE_SWIGLU), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = backward(inp, f, workspace=ws)
    for _ in range(2):
        ws.fill_(0xFF)
        graph.replay()
        for k in ("dx", "dgamma", "dw1", "dw2", "db1", "db2", "dh"):
            assert torch.equal(g[k], ref[k]), k


def test_no_tokens_and_refusals():
    inp = inputs("gpt_ln_mlp_bwd", None, 16, 64, 96)
    f = forward(inp, None, True)
    for k in ("x", "dy"):
        inp[k] = inp[k][:0]
    inp["M"] = 0
    e = {k: v[:0] if k in ("codes", "ln", "mu", "rs", "scales") else v for k, v in f.items()}
    g = backward(inp, e)
    torch.cuda.synchronize()
    for k in ("dgamma", "dbeta", "dw1", "dw2", "db1", "db2"):
        assert (g[k] == 0).all(), k
    inp = inputs("gpt_ln_mlp_bwd", None, 16, 64, 96)
    with pytest.raises(ValueError, match="h_codes"):
        backward(inp, dict(f, codes=f["codes"][:8]))
    inp = inputs("gpt_ln_mlp_bwd", None, 16, 64, 48)  # half a block
    with pytest.raises((te.TEError, ValueError)):
        forward(inp, None, True)
    b = te.binding
    P = 4096
    call = lambda F, codes: te.lib().te_layernorm_mlp_fwd_ckpt(
        P, P, P, P, P, b.TE_BF16, None, None, b.TE_LAYERNORM, 0, 1e-6, b.TE_GELU, None, 16, 64, F, b.TE_BF16, P, codes, P,
        None, None, None, None, P, 1 << 30, None)
    assert call(48, P) == b.TE_ERR_UNSUPPORTED
    assert call(64, None) == b.TE_ERR_INVALID_ARG
    assert call(64, P + 8) == b.TE_ERR_UNSUPPORTED


def test_difference_to_the_uncompressed_gradients_is_the_checkpoints_rounding():
    """The block's loss gradient against the one from saved_h: h moves by at most 2^-4 of itself (E4M3) or
    half of E4M3's smallest step (2^-10) of its block's scale, so act(h) and act'(h) move with it."""
    inp = inputs("gpt_ln_mlp_bwd", None, 256, 256, 512)
    a, f = forward(inp, None, False), forward(inp, None, True)
    h = np64(a["h"])
    hq = bs.unpack(*bs.pack(h, "mxfp8"), "mxfp8")
    step = np.ldexp(1.0, np.frexp(np.abs(h).reshape(256, -1, 32).max(-1) / 448.0)[1]).repeat(32, -1)
    assert (np.abs(h - hq) <= np.maximum(np.abs(h) / 16, step * 2.0 ** -10)).all()
    g = backward(inp, f)
    da = np64(inp["dy"]) @ np64(inp["w2"]).T
    lip = np.abs(ob.act_bwd(np.ones_like(h), h + 1e-3, "gelu") - ob.act_bwd(np.ones_like(h), h - 1e-3, "gelu")).max() / 2e-3
    bound = np.abs(da) * (lip * 1.5 * np.abs(h - hq)) + 2.0 ** -7 * np.abs(da) * 1.2 + 2e-2
    assert (np.abs(np64(g["dh"]) - ob.act_bwd(da, h, "gelu")) <= bound).all()


def test_tensors_the_binding_refuses():
    """Another device, type or size of any argument is an error on the host."""
    inp = inputs("gpt_ln_mlp_bwd", None, 16, 64, 96)
    for mode in (None, "delayed"):
        f = forward(inp, mode, True)
        for k in ("x", "gamma", "beta", "w1", "w2"):
            for bad in (inp[k].cpu(), inp[k].double(), torch.cat([inp[k], inp[k]])):
                if k == "x" and bad.shape != inp[k].shape:
                    continue  # another number of rows is another call
                with pytest.raises((ValueError, KeyError)):
                    forward(dict(inp, **{k: bad}), mode, True)
        for k in ("ln", "mu", "rs", "codes", "scales"):
            for bad in (f[k].cpu(), f[k].double(), f[k][:8].contiguous()):
                with pytest.raises(ValueError):
                    backward(inp, dict(f, **{k: bad}))
        with pytest.raises(ValueError):
            backward(dict(inp, dy=inp["dy"][:8].contiguous()), f)
        with pytest.raises(ValueError):
            backward(inp, f, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    host = te.Quantizer(2.0, device="cpu")
    with pytest.raises(ValueError, match="grad.scale"):
        backward(inp, dict(f, qs=te.QuantizerSet(**dict(vars(f["qs"]), grad=host))))
    F = inp["F"]
    c = te.block_empty("mxfp8", 16, F)
    dy = torch.zeros(16, F, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="q.scale"):
        te.te_dact_dbias_ckpt(dy, *c, "gelu", torch.empty(16, F, dtype=torch.uint8, device=DEV), q=host)


def test_workspaces_of_any_type_that_are_dense():
    """A workspace counts by its bytes whatever its type; one without that many behind it is refused."""
    inp = inputs("gpt_ln_mlp_bwd", None, 48, 128, 96)
    f = forward(inp, None, True)
    ref = backward(inp, f)
    b = te.binding
    kw = dict(norm_type=inp["norm"], activation_type=inp["act"], epsilon=inp["eps"])
    args = (inp["x"], inp["gamma"], inp["beta"], inp["w1"], inp["w2"], inp["b1"], inp["b2"])
    size = lambda op: te.workspace_size(op, 48, 128, 96, b.TE_BF16, False, b.TE_BF16, b.TE_GELU)
    bad = torch.empty(1, dtype=torch.uint8, device=DEV).expand(size(b.TE_OP_LAYERNORM_MLP_BWD) + (1 << 20))
    for dt in (torch.uint8, torch.float32, torch.int64):
        new = lambda op: torch.empty((size(op) + 7) // 8 * 8 // torch.empty(0, dtype=dt).element_size(), dtype=dt, device=DEV)
        out, c = torch.empty_like(f["out"]), te.block_empty("mxfp8", 48, 96)
        te.te_layernorm_mlp_fwd_ckpt(*args, out, *c, workspace=new(b.TE_OP_LAYERNORM_MLP_FWD), **kw)
        assert torch.equal(out, f["out"]) and torch.equal(c[0], f["codes"])
        g = backward(inp, f, workspace=new(b.TE_OP_LAYERNORM_MLP_BWD))
        for k in ("dx", "dgamma", "dw1", "dw2", "db1", "db2"):
            assert torch.equal(g[k], ref[k]), (dt, k)
    with pytest.raises(ValueError, match="workspace"):
        te.te_layernorm_mlp_fwd_ckpt(*args, out, *c, workspace=bad, **kw)
    with pytest.raises(ValueError, match="workspace"):
        backward(inp, f, workspace=bad)


def test_on_streams_of_their_own():
    """Forward and backward on a passed stream and on a current one, without a workspace of the caller's."""
    inp = inputs("llama_rms_mlp", None, 200, 256, 288)
    ref = forward(inp, None, True)
    want = backward(inp, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (inp["x"], inp["gamma"], inp["beta"], inp["w1"], inp["w2"], None, None)
    kw = dict(norm_type=inp["norm"], zero_centered_gamma=inp["zero_centered_gamma"], activation_type=inp["act"],
              epsilon=inp["eps"])
    got = []
    for passed in (True, False, True, False):
        f = dict(ref, out=torch.empty_like(ref["out"]), ln=torch.empty_like(ref["ln"]), mu=torch.empty_like(ref["mu"]),
                 rs=torch.empty_like(ref["rs"]))
        f["codes"], f["scales"] = te.block_empty("mxfp8", 200, 576)
        call = lambda **st: (te.te_layernorm_mlp_fwd_ckpt(*args, f["out"], f["codes"], f["scales"], saved_ln_out=f["ln"],
                                                          mu=f["mu"], rsigma=f["rs"], **kw, **st), backward(inp, f, **st))[1]
        s.wait_stream(torch.cuda.current_stream())
        if passed:
            got.append(call(stream=s))
            torch.empty(1 << 21, dtype=torch.uint8, device=DEV).fill_(255)  # would land in a workspace freed too early
        else:
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    assert te.get_device_status() == 0
    for g in got:
        for k in ("out", "codes", "scales", "dx", "dgamma", "dw1", "dw2", "db1", "db2", "dh"):
            assert torch.equal(g[k], want[k]), k

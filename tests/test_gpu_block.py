"""The block around the layer (block.py) on the GPU against the oracles
chained in float64: a training step forward and backward, and a decode step
with 4-bit experts, also as a CUDA graph.

Routing is discrete, so both sides route by the logits that the GPU computed;
every other value is the oracle's own.  The errors of a chain of bf16 stages
are those of the layer's own parity tests: normwise 2e-2.
"""
import pytest
import torch

import mixture_experts_token_gb300 as moe
from mixture_experts_token_gb300 import block
from oracle import block_ref, moe_ref
from tests.gpu_util import TOL, f64, normwise

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _weights(c, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16

    def normal(*shape, std=0.05, mean=0.0, t=dt):
        return (torch.randn(*shape, generator=g) * std + mean).to(t).cuda()
    f = torch.float32
    w = {n: normal(c.H, std=0.2, mean=1.0, t=f)
         for n in ("w_pre", "w_post", "w_next")}
    w["w_router"] = normal(c.H, c.E, std=0.1)
    w["w_gate"], w["w_up"] = normal(c.E, c.H, c.F), normal(c.E, c.H, c.F)
    w["w_down"] = normal(c.E, c.F, c.H)
    return w, normal


def _layer(c, h, logits, w):
    """Oracle forward of the dropless layer."""
    cfg = moe_ref.MoEConfig(c.T, c.H, c.E, c.k, c.F, c.S, -1.0)
    return moe_ref.layer_dropless(cfg, h, logits, moe_ref.dense_weights(
        w["w_gate"], w["w_up"], w["w_down"])).y


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
def test_training_step(dtype, kind):
    T, H, E, k, F = 70, 128, 4, 2, 128
    c = moe.make_config(T, H, E, k, F, 2, -1.0, dtype=dtype)
    o = moe.make_block_norm(EPS, 0.0, 0.8, ("none", "token", "channel",
                                            "full").index(kind))
    w, normal = _weights(c, dtype)
    x = normal(T, H, std=2.0)
    gate = {"none": lambda: None,
            "token": lambda: normal(T, std=1.0, t=torch.float32),
            "channel": lambda: normal(H, std=1.0, t=torch.float32),
            "full": lambda: normal(T, H, std=1.0)}[kind]()
    dout, dh = normal(T, H, std=1.0), normal(T, H, std=1.0)
    b = block.TrainBlock(c, o, w)
    out, h_next = b.forward(x, gate)
    got = b.backward(dout, dh)
    torch.cuda.synchronize()
    assert b.status.item() == 0

    W = {n: f64(v) for n, v in w.items()}
    g64 = None if gate is None else f64(gate)
    logits = b.logits.cpu().numpy()
    h = block_ref.norm(f64(x), W["w_pre"], EPS)
    y = _layer(c, h, logits, W)
    want, _ = block_ref.block_out(f64(x), y, W["w_post"], g64, kind, EPS,
                                  0.0, 0.8)
    assert normwise(f64(out), want) <= TOL[dtype]
    assert normwise(f64(h_next), block_ref.norm(want, W["w_next"], EPS)) \
        <= TOL[dtype]
    back = {n: v for n, (v, _) in block_ref.block_out_backward(
        y, W["w_post"], g64, kind, want, W["w_next"], f64(dout), f64(dh),
        EPS, 0.0, 0.8).items()}
    cfg = moe_ref.MoEConfig(T, H, E, k, F, 2, -1.0)
    lay = moe_ref.layer_backward_dropless(
        cfg, h, logits, W["w_gate"], W["w_up"], W["w_down"], back["dy"])
    dhid = lay.dx + lay.dlogits @ W["w_router"].T
    dx, dw_pre, _, _ = block_ref.norm_backward(f64(x), W["w_pre"], dhid, EPS)
    expect = {"dx": dx + back["dx"], "w_pre": dw_pre,
              "w_post": back["dw_post"], "w_next": back["dw_next"],
              "w_router": h.T @ lay.dlogits, "w_gate": lay.dwg,
              "w_up": lay.dwu, "w_down": lay.dwd}
    if gate is not None:
        expect["gate"] = back["dgate"]
    for n, v in expect.items():
        assert normwise(f64(got[n]), v) <= TOL[dtype], n


@pytest.mark.parametrize("T,H,E,k,F,dtype", [
    (1, 256, 16, 4, 136, "bf16"), (9, 520, 7, 3, 264, "bf16"),
    (5, 132, 6, 2, 68, "f32")])
@pytest.mark.parametrize("zeros", [False, True])
def test_decode_step(T, H, E, k, F, dtype, zeros):
    c = moe.make_config(T, H, E, k, F, 1, dtype=dtype)
    o = moe.make_block_norm(EPS, 1.0, 1.0, moe.MOE_GATE_CHANNEL)
    w4 = moe.make_w4(64, zeros)
    w, normal = _weights(c, dtype, seed=1)
    dense = {}
    for n in ("w_gate", "w_up", "w_down"):
        q = block.quantize_experts(w4, w[n])
        back = torch.empty_like(w[n], dtype=torch.float32)
        moe.moe_w4_dequantize(w4, *w[n].shape, q, back)
        # a step of the group's range, over 15 or 14 steps
        w32 = w[n].float()
        assert (back - w32).abs().max() <= 0.1 * w32.abs().max()
        w[n], dense[n] = q, f64(back)
    x = normal(T, H, std=2.0)
    gate = normal(H, std=1.0, t=torch.float32)
    b = block.DecodeBlock(c, o, w4, w)
    out, h_next = b.step(x, gate)
    torch.cuda.synchronize()
    assert b.b["status"].item() == 0
    W = {n: f64(w[n]) for n in ("w_pre", "w_post", "w_next")}
    h = block_ref.norm(f64(x), W["w_pre"], EPS, 1.0)
    y = _layer(c, h, b.logits.cpu().numpy(), dense)
    want, _ = block_ref.block_out(f64(x), y, W["w_post"], f64(gate),
                                  "channel", EPS, 1.0, 1.0)
    assert normwise(f64(out), want) <= TOL[dtype]
    assert normwise(f64(h_next),
                    block_ref.norm(want, W["w_next"], EPS, 1.0)) <= TOL[dtype]

    # the same step as a graph, on other rows
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(x, gate)
    x2 = normal(T, H, std=2.0)
    kept = x.clone()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(b.out, first)
    x.copy_(kept)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, first)


@pytest.mark.parametrize("post,nxt", [(False, True), (True, False),
                                      (False, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_without_a_norm(dtype, post, nxt):
    """w_post, w_next or both absent, in the training and the decode step."""
    T, H, E, k, F = 9, 128, 4, 2, 128
    c = moe.make_config(T, H, E, k, F, 1, -1.0, dtype=dtype)
    o = moe.make_block_norm(EPS, 0.0, 0.8, moe.MOE_GATE_CHANNEL)
    w, normal = _weights(c, dtype, seed=2)
    for n, there in (("w_post", post), ("w_next", nxt)):
        if not there:
            w[n] = None
    x, gate = normal(T, H, std=2.0), normal(H, std=1.0, t=torch.float32)
    dout, dh = normal(T, H, std=1.0), normal(T, H, std=1.0) if nxt else None

    def check_forward(b, out, h_next, W):
        h = block_ref.norm(f64(x), W["w_pre"], EPS)
        y = _layer(c, h, b.logits.cpu().numpy(), W)
        want, _ = block_ref.block_out(f64(x), y, W["w_post"], f64(gate),
                                      "channel", EPS, 0.0, 0.8)
        assert normwise(f64(out), want) <= TOL[dtype]
        if nxt:
            assert normwise(f64(h_next), block_ref.norm(
                want, W["w_next"], EPS)) <= TOL[dtype]
        else:
            assert h_next is None
        return h, y, want

    W = {n: None if v is None else f64(v) for n, v in w.items()}
    b = block.TrainBlock(c, o, w)
    h, y, want = check_forward(b, *b.forward(x, gate), W)
    got = b.backward(dout, dh)
    back = {n: v for n, (v, _) in block_ref.block_out_backward(
        y, W["w_post"], f64(gate), "channel", want, W["w_next"], f64(dout),
        f64(dh) if nxt else None, EPS, 0.0, 0.8).items()}
    lay = moe_ref.layer_backward_dropless(
        moe_ref.MoEConfig(T, H, E, k, F, 1, -1.0), h, b.logits.cpu().numpy(),
        W["w_gate"], W["w_up"], W["w_down"], back["dy"])
    dx, dw_pre, _, _ = block_ref.norm_backward(
        f64(x), W["w_pre"], lay.dx + lay.dlogits @ W["w_router"].T, EPS)
    expect = {"dx": dx + back["dx"], "w_pre": dw_pre, "gate": back["dgate"],
              "w_down": lay.dwd}
    for n in ("w_post", "w_next"):
        if w[n] is None:
            assert got[n] is None
        else:
            expect[n] = back["d" + n]
    for n, v in expect.items():
        assert normwise(f64(got[n]), v) <= TOL[dtype], n

    w4 = moe.make_w4(64, True)
    for n in ("w_gate", "w_up", "w_down"):
        q = block.quantize_experts(w4, w[n])
        full = torch.empty_like(w[n], dtype=torch.float32)
        moe.moe_w4_dequantize(w4, *w[n].shape, q, full)
        w[n], W[n] = q, f64(full)
    b = block.DecodeBlock(c, o, w4, w)
    check_forward(b, *b.step(x, gate), W)


def test_training_step_without_tokens():
    """T = 0: no rows come out and every weight's gradient is zero."""
    c = moe.make_config(0, 128, 4, 2, 128, 1, -1.0)
    o = moe.make_block_norm(EPS, 0.0, 1.0, moe.MOE_GATE_CHANNEL)
    w, normal = _weights(c, "bf16", seed=3)
    x, gate = normal(0, 128), normal(128, t=torch.float32)
    b = block.TrainBlock(c, o, w)
    out, h_next = b.forward(x, gate)
    got = b.backward(x.clone(), x.clone())
    torch.cuda.synchronize()
    assert out.shape == h_next.shape == got["dx"].shape == (0, 128)
    for n in ("gate", "w_router", *(n for n in w)):
        assert (got[n] == 0).all(), n

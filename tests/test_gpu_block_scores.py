"""block.py with routing by scores, and with microscaled experts, on the GPU:
a training step's outputs and gradients against the same formulas under
float64 automatic differentiation, and a decode step against float64 on the
weights' quantised values, also as a CUDA graph.

Routing is discrete, so both sides take the experts that the GPU chose (their
choice itself is tested against the oracle); every other value is the
reference's own, rows and activations rounded to 4 bits where the step rounds
them (the rows from the norm's stored values).  The errors of a chain of bf16
stages are those of the layer's own parity tests: normwise 2e-2, far above what
the few activations may do that lie so near the middle of two codes that
float32 and float64 round them apart.
"""
import pytest
import torch

import mixture_experts_token_gb300 as moe
from mixture_experts_token_gb300 import block
from oracle import mx_ref, route_ref
from tests.gpu_util import TOL, f64, normwise
from tests.test_gpu_block import _weights

pytestmark = pytest.mark.gpu

EPS = 1e-6


def t64(t):
    return t.detach().cpu().double()


def norm(v, w):
    return v * (v.square().mean(1, keepdim=True) + EPS).rsqrt() * w


def layer(h, idx, weights, w):
    """Dropless layer in float64: the chosen experts' FFNs, weighted."""
    rows = []
    for t in range(len(h)):
        y = 0
        for j, e in enumerate(idx[t].tolist()):
            g, u = h[t] @ w["w_gate"][e], h[t] @ w["w_up"][e]
            y = y + weights[t, j] * ((g * torch.sigmoid(g) * u)
                                     @ w["w_down"][e])
        rows.append(y)
    return torch.stack(rows)


def on_grid(v, size, scale):
    q = mx_ref.quantize_rows(v.float().numpy(), size, scale)
    return torch.from_numpy(mx_ref.dequantize_rows(*q, size, scale))


def mx_layer(h, idx, weights, w, mx):
    """The layer with rows and activations rounded to 4 bits."""
    x = on_grid(h, mx.block, mx.x_scale)
    y = torch.zeros(len(h), w["w_down"].shape[2], dtype=torch.float64)
    for j in range(idx.shape[1]):
        for e in range(len(w["w_gate"])):
            t = idx[:, j] == e
            if t.any():
                g, u = x[t] @ w["w_gate"][e], x[t] @ w["w_up"][e]
                a = on_grid(g * torch.sigmoid(g) * u, mx.block, mx.h_scale)
                y[t] += weights[t, j, None] * (a @ w["w_down"][e])
    return y


def weigh(logits, idx, sigmoid, renorm, scale):
    s = torch.sigmoid(logits) if sigmoid else logits.softmax(1)
    s = s.gather(1, idx)
    return scale * (s / s.sum(1, keepdim=True) if renorm else s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score,renorm", [
    (moe.MOE_SCORE_SIGMOID, True), (moe.MOE_SCORE_SOFTMAX, False),
    (moe.MOE_SCORE_SOFTMAX, True)])
def test_training_step(dtype, score, renorm):
    T, H, E, k, F = 30, 128, 8, 3, 128
    sigmoid = score == moe.MOE_SCORE_SIGMOID
    c = moe.make_config(T, H, E, k, F, 2, -1.0, dtype=dtype)
    o = moe.make_block_norm(EPS, 0.0, 0.8)
    r = moe.make_route_scores(score, 4, 2, 2, renorm, 2.5)
    w, normal = _weights(c, dtype)
    bias = normal(E, std=0.1, t=torch.float32)
    x, dout, dh = (normal(T, H, std=s) for s in (2.0, 1.0, 1.0))
    b = block.TrainBlock(c, o, w, route=r, bias=bias)
    out, h_next = b.forward(x)
    got = b.backward(dout, dh)
    torch.cuda.synchronize()
    assert b.status.item() == 0

    idx = b.b["topk_idx"].cpu().long()
    want, _ = route_ref.route(b.logits.cpu().numpy(), bias.cpu().numpy(), k,
                              sigmoid, 4, 2, 2, renorm, 2.5)
    assert (idx.numpy() == want).all()
    W = {n: t64(v).requires_grad_() for n, v in w.items()}
    x64 = t64(x).requires_grad_()
    h = norm(x64, W["w_pre"])
    y = layer(h, idx, weigh(h @ W["w_router"], idx, sigmoid, renorm, 2.5), W)
    o64 = 0.8 * x64 + norm(y, W["w_post"])
    n64 = norm(o64, W["w_next"])
    ((o64 * t64(dout)).sum() + (n64 * t64(dh)).sum()).backward()
    assert normwise(f64(out), o64.detach().numpy()) <= TOL[dtype]
    assert normwise(f64(h_next), n64.detach().numpy()) <= TOL[dtype]
    assert normwise(f64(got["dx"]), x64.grad.numpy()) <= TOL[dtype]
    for n in W:
        assert normwise(f64(got[n]), W[n].grad.numpy()) <= TOL[dtype], n


@pytest.mark.parametrize("T,H,E,k,F,dtype", [
    (1, 256, 16, 4, 160, "bf16"), (9, 544, 8, 3, 288, "bf16"),
    (5, 160, 6, 2, 96, "f32"), (70, 256, 8, 2, 128, "bf16")])
@pytest.mark.parametrize("size", [16, 32])
def test_decode_step(T, H, E, k, F, dtype, size):
    c = moe.make_config(T, H, E, k, F, 1, dtype=dtype)
    o = moe.make_block_norm(EPS)
    r = moe.make_route_scores(moe.MOE_SCORE_SIGMOID, 2, 1, 2, True, 1.5)
    mx = moe.make_mx(size, *((0.004, 0.002) if size == 16 else ()))
    w, normal = _weights(c, dtype, seed=1)
    dense = {}
    for n in ("w_gate", "w_up", "w_down"):
        q, scale = block.quantize_experts_mx(mx, w[n])
        back = torch.empty_like(w[n], dtype=torch.float32)
        moe.moe_mx_dequantize(mx, *w[n].shape, q, scale, back)
        # half a step of codes at most, 1/6 of a block's largest magnitude
        # (blocks of 32: up to 1/4, where it is cut from 8 to 6)
        w32 = w[n].float()
        assert (back - w32).abs().max() <= 0.26 * w32.abs().max()
        w[n], w[n + "_scale"], dense[n] = q, scale, t64(back)
    bias = normal(E, std=0.05, t=torch.float32)
    x = normal(T, H, std=2.0)
    b = block.DecodeBlock(c, o, mx, w, route=r, bias=bias)
    out, h_next = b.step(x)
    torch.cuda.synchronize()
    assert b.b["status"].item() == 0
    idx = b.b["topk_idx"].cpu().long()
    want, ww = route_ref.route(b.logits.cpu().numpy(), bias.cpu().numpy(), k,
                               True, 2, 1, 2, True, 1.5)
    assert (idx.numpy() == want).all()
    assert normwise(f64(b.h), norm(t64(x), t64(w["w_pre"])).numpy()) \
        <= TOL[dtype]
    y = mx_layer(t64(b.h), idx, torch.from_numpy(ww), dense, mx)
    o64 = t64(x) + norm(y, t64(w["w_post"]))
    assert normwise(f64(out) - f64(x), (o64 - t64(x)).numpy()) <= 2e-2
    assert normwise(f64(h_next), norm(t64(out), t64(w["w_next"])).numpy()) \
        <= TOL[dtype]

    want = [out.clone(), h_next.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(x)
    x0 = x.clone()
    x.copy_(normal(T, H, std=2.0))
    graph.replay()
    x.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want[0]) and torch.equal(b.h_next, want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_weights_that_are_not_finite_spoil_their_block_alone(dtype, bad):
    g = torch.Generator().manual_seed(5)
    w = (torch.randn(3, 96, 40, generator=g) * 0.02).to(dtype).cuda()
    mx = moe.make_mx(16)
    clean, scale = block.quantize_experts_mx(mx, w)
    broken = w.clone()
    broken[1, 35, 7] = float(bad)
    q, s = block.quantize_experts_mx(mx, broken)
    assert torch.equal(s, scale)
    a, b = (torch.empty_like(w, dtype=torch.float32) for _ in range(2))
    moe.moe_mx_dequantize(mx, *w.shape, clean, scale, a)
    moe.moe_mx_dequantize(mx, *w.shape, q, s, b)
    assert b[1, 32:48, 7].isnan().all()
    b[1, 32:48, 7] = a[1, 32:48, 7]
    assert torch.equal(a, b)

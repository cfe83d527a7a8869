"""The block-norm oracle's gradients against central differences (CPU)."""
import numpy as np
import pytest

from oracle import block_ref as ref

EPS = 1e-6


def _case(kind, post, nxt, seed=0, T=3, H=8):
    g = np.random.default_rng(seed)
    gate = {"none": None, "token": g.normal(size=T),
            "channel": g.normal(size=H), "full": g.normal(size=(T, H))}[kind]
    return dict(x=g.normal(size=(T, H)), y=g.normal(size=(T, H)),
                w_post=g.normal(size=H) if post else None, gate=gate,
                w_next=g.normal(size=H) if nxt else None,
                dout=g.normal(size=(T, H)),
                dh=g.normal(size=(T, H)) if nxt else None)


def _loss(c, kind):
    out, _ = ref.block_out(c["x"], c["y"], c["w_post"], c["gate"], kind, EPS,
                           1.0, 0.7)
    loss = (c["dout"] * out).sum()
    if c["w_next"] is not None:
        loss += (c["dh"] * ref.norm(out, c["w_next"], EPS, 1.0)).sum()
    return loss


@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("nxt", [False, True])
def test_gradients_match_differences(kind, post, nxt):
    c = _case(kind, post, nxt)
    out, _ = ref.block_out(c["x"], c["y"], c["w_post"], c["gate"], kind, EPS,
                           1.0, 0.7)
    got = ref.block_out_backward(c["y"], c["w_post"], c["gate"], kind, out,
                                 c["w_next"], c["dout"], c["dh"], EPS, 1.0,
                                 0.7)
    names = {"dx": "x", "dy": "y", "dw_post": "w_post", "dgate": "gate",
             "dw_next": "w_next"}
    step = 1e-5   # error of a central difference: step^2 and 1e-16/step
    for grad, name in names.items():
        if c[name] is None:
            continue
        want = np.empty_like(c[name])
        for i in np.ndindex(c[name].shape):
            old = c[name][i]
            c[name][i] = old + step
            up = _loss(c, kind)
            c[name][i] = old - step
            want[i] = (up - _loss(c, kind)) / (2 * step)
            c[name][i] = old
        assert np.allclose(got[grad][0], want, rtol=1e-6, atol=1e-7), grad
        assert np.all(np.abs(got[grad][0]) <= got[grad][1] * (1 + 1e-12))


def test_magnitudes_bound_a_float32_evaluation():
    c = _case("channel", True, True, seed=3, T=7, H=64)
    out, _ = ref.block_out(c["x"], c["y"], c["w_post"], c["gate"], "channel",
                           EPS)
    args = (c["y"], c["w_post"], c["gate"], "channel", out, c["w_next"],
            c["dout"], c["dh"], EPS)
    want = ref.block_out_backward(*args)
    got = ref.block_out_backward(*(a.astype(np.float32)
                                   if isinstance(a, np.ndarray) else a
                                   for a in args))
    for name, (v, mag) in want.items():
        # inputs rounded to 2^-24 each, a handful of them a term
        assert np.all(np.abs(got[name][0] - v) <= 64 * 2.0 ** -24 * mag), name

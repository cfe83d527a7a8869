"""What block.py does before any launch: its buffers and refusals (CPU)."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import mixture_experts_token_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from mixture_experts_token_gb300 import build
        build.build()
    return m


def weights(H, E, F, w_post=True, w_next=True):
    col = lambda on: torch.ones(H) if on else None  # noqa: E731
    bf = dict(dtype=torch.bfloat16)
    return dict(w_pre=torch.ones(H), w_post=col(w_post), w_next=col(w_next),
                w_router=torch.zeros(H, E, **bf),
                w_gate=torch.zeros(E, H, F, **bf),
                w_up=torch.zeros(E, H, F, **bf),
                w_down=torch.zeros(E, F, H, **bf))


def packed(m, w4, w):
    """The same weights with the experts' in (unwritten) 4-bit buffers."""
    return {**w, **{n: m.alloc_w4(w4, *w[n].shape, "cpu")
                    for n in ("w_gate", "w_up", "w_down")}}


@pytest.mark.parametrize("w_next", [True, False])
def test_a_block_without_a_following_norm_has_no_rows_of_it(m, w_next):
    """Nothing writes h_next then, so there is nothing to hand out."""
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    w = weights(64, 4, 32, w_next=w_next)
    o, w4 = m.make_block_norm(), m.make_w4(32)
    for b in (block.TrainBlock(c, o, w, device="cpu"),
              block.DecodeBlock(c, o, w4, packed(m, w4, w), device="cpu")):
        assert (b.h_next is not None) == w_next, type(b).__name__


def test_quantizing_a_transposed_view_is_refused(m):
    """Weights stored [E, N, K] and seen as [E, K, N]: their elements do not
    lie where the quantiser reads them."""
    from mixture_experts_token_gb300 import block
    w = torch.zeros(2, 48, 64, dtype=torch.bfloat16)
    for view in (w.transpose(1, 2), w[:, :, ::2], w):    # the last: no GPU
        with pytest.raises(ValueError, match="w: needs"):
            block.quantize_experts(m.make_w4(32), view)


def wrong(t):
    """Tensors that a kernel would misread in the place of t."""
    yield torch.zeros(*t.shape, 2, dtype=t.dtype)[..., 0]       # strided
    if t.dim() > 1:
        yield torch.zeros(t.shape[::-1], dtype=t.dtype).permute(
            *reversed(range(t.dim())))                          # transposed
    yield torch.zeros(t.numel() + 8, dtype=t.dtype)             # too long
    yield t.to(torch.float64)
    yield t.to("meta")


@pytest.mark.parametrize("name", ["w_pre", "w_post", "w_next", "w_router",
                                  "w_gate", "w_up", "w_down"])
def test_blocks_refuse_weights_they_would_misread(m, name):
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    o, w4, w = m.make_block_norm(), m.make_w4(32), weights(64, 4, 32)
    q = packed(m, w4, w)
    for bad in wrong(w[name]):
        with pytest.raises(ValueError, match=name):
            block.TrainBlock(c, o, {**w, name: bad}, device="cpu")
    for bad in wrong(q[name]):
        with pytest.raises(ValueError, match=name):
            block.DecodeBlock(c, o, w4, {**q, name: bad}, device="cpu")
    if name in ("w_gate", "w_up", "w_down"):     # not quantised
        with pytest.raises(ValueError, match=name):
            block.DecodeBlock(c, o, w4, {**q, name: w[name]}, device="cpu")
    for bad in wrong(torch.zeros(3, 4)):
        with pytest.raises(ValueError, match="logit_offset"):
            block.TrainBlock(c, o, w, bad, device="cpu")
        with pytest.raises(ValueError, match="logit_offset"):
            block.DecodeBlock(c, o, w4, q, bad, device="cpu")


@pytest.mark.parametrize("kind,shape,dtype", [
    (1, (3,), torch.float32), (2, (64,), torch.float32),
    (3, (3, 64), torch.bfloat16)])
def test_steps_refuse_rows_and_gates_they_would_misread(m, kind, shape,
                                                        dtype):
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    o, w4, w = m.make_block_norm(gate=kind), m.make_w4(32), weights(64, 4, 32)
    train = block.TrainBlock(c, o, w, device="cpu")
    decode = block.DecodeBlock(c, o, w4, packed(m, w4, w), device="cpu")
    x, gate = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(
        shape, dtype=dtype)
    for bad in wrong(x):
        for call in (lambda: train.forward(bad, gate),
                     lambda: decode.step(bad, gate)):
            with pytest.raises(ValueError, match="x: needs"):
                call()
        with pytest.raises(ValueError, match="dout"):
            train.backward(bad)
        with pytest.raises(ValueError, match="dh_next"):
            train.backward(x, bad)
    for bad in wrong(gate):
        for call in (lambda: train.forward(x, bad),
                     lambda: decode.step(x, bad)):
            with pytest.raises(ValueError, match="gate"):
                call()


@pytest.mark.parametrize("kind", [-1, 4])
def test_an_unknown_gate_is_the_librarys_error(m, kind):
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    b = block.TrainBlock(c, m.make_block_norm(gate=kind), weights(64, 4, 32),
                         device="cpu")
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(m.MoeError) as err:
        b.forward(x, x)
    assert err.value.status == m.MOE_ERR_INVALID_ARG

"""What block.py does before any launch with routing by scores and with
microscaled experts: its buffers and refusals (CPU)."""
import os

import pytest
import torch

from tests.test_block_host import weights, wrong


@pytest.fixture(scope="module")
def m():
    import mixture_experts_token_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from mixture_experts_token_gb300 import build
        build.build()
    return m


def mx_weights(m, mx, w):
    return {**w, **{n: m.alloc_mx(mx, *w[n].shape, "cpu")
                    for n in ("w_gate", "w_up", "w_down")}}


@pytest.mark.parametrize("block_size", [16, 32])
def test_blocks_refuse_a_bias_and_scales_they_would_misread(m, block_size):
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    o, r, w = m.make_block_norm(), m.make_route_scores(), weights(64, 4, 32)
    mx = m.make_mx(block_size)
    q = mx_weights(m, mx, w)
    made = block.DecodeBlock(c, o, mx, q, device="cpu", route=r,
                             bias=torch.zeros(4))
    assert made.ws.numel() >= m.moe_mx_workspace_bytes(c, mx) > 0
    for bad in wrong(torch.zeros(4)):
        with pytest.raises(ValueError, match="bias"):
            block.TrainBlock(c, o, w, device="cpu", route=r, bias=bad)
        with pytest.raises(ValueError, match="bias"):
            block.DecodeBlock(c, o, mx, q, device="cpu", route=r, bias=bad)
        for n in ("w_gate", "w_up", "w_down"):
            with pytest.raises(ValueError, match=n + "_scale"):
                block.DecodeBlock(c, o, mx, {**q, n + "_scale": bad},
                                  device="cpu")
    with pytest.raises(ValueError, match="bias"):       # nobody to add it
        block.TrainBlock(c, o, w, device="cpu", bias=torch.zeros(4))
    for n in ("w_gate", "w_up", "w_down"):
        for bad in wrong(q[n]):
            with pytest.raises(ValueError, match=n):
                block.DecodeBlock(c, o, mx, {**q, n: bad}, device="cpu")


def test_scales_belong_to_microscaled_experts(m):
    from mixture_experts_token_gb300 import block
    c, w4 = m.make_config(3, 64, 4, 2, 32, 1), m.make_w4(32)
    w = weights(64, 4, 32)
    q = {**w, **{n: m.alloc_w4(w4, *w[n].shape, "cpu")
                 for n in ("w_gate", "w_up", "w_down")}}
    with pytest.raises(ValueError, match="w_up_scale"):
        block.DecodeBlock(c, m.make_block_norm(), w4,
                          {**q, "w_up_scale": torch.ones(4)}, device="cpu")


def test_experts_are_given_by_name_as_before(m):
    from mixture_experts_token_gb300 import block
    c, o, w4 = m.make_config(3, 64, 4, 2, 32, 1), m.make_block_norm(), \
        m.make_w4(32)
    w = weights(64, 4, 32)
    q = {**w, **{n: m.alloc_w4(w4, *w[n].shape, "cpu")
                 for n in ("w_gate", "w_up", "w_down")}}
    made = block.DecodeBlock(cfg=c, opt=o, w4=w4, weights=q, device="cpu")
    assert made.w4 is w4
    mx = m.make_mx(32)
    made = block.DecodeBlock(cfg=c, opt=o, w4=mx, weights=mx_weights(m, mx, w),
                             device="cpu")
    assert made.w4 is mx


def test_a_capped_pass_is_the_layers(m):
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    with pytest.raises(ValueError, match="capped"):
        block.TrainBlock(c, m.make_block_norm(), weights(64, 4, 32),
                         mode=m.MOE_MODE_CAPPED, device="cpu",
                         route=m.make_route_scores())


def test_quantizing_a_transposed_view_is_refused(m):
    from mixture_experts_token_gb300 import block
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    for view in (w.transpose(1, 2), w[:, :, ::2], w):    # the last: no GPU
        with pytest.raises(ValueError, match="w: needs"):
            block.quantize_experts_mx(m.make_mx(32), view)

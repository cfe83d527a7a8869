"""What block.py does before any launch: its buffers (CPU)."""
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


@pytest.mark.parametrize("w_next", [True, False])
def test_a_block_without_a_following_norm_has_no_rows_of_it(m, w_next):
    """Nothing writes h_next then, so there is nothing to hand out."""
    from mixture_experts_token_gb300 import block
    c = m.make_config(3, 64, 4, 2, 32, 1)
    w = weights(64, 4, 32, w_next=w_next)
    o, w4 = m.make_block_norm(), m.make_w4(32)
    for b in (block.TrainBlock(c, o, w, device="cpu"),
              block.DecodeBlock(c, o, w4, w, device="cpu")):
        assert (b.h_next is not None) == w_next, type(b).__name__

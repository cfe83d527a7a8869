"""Routing by scores, a bias and groups on the GPU against the float64 oracle.

Choices are whole numbers and equal the oracle's.  A weight is a quotient of
float32 exponentials (two ulps) and a sum of at most 32 of them: 16 roundings
of 2^-24 in all, 1e-6 of it.  A gradient is a weight times what is left of a
sum of at most 32 terms: 1e-6 of the sum of its terms' magnitudes, doubled for
the softmax's own sum of up to 1024.
"""
import numpy as np
import pytest
import torch

import mixture_experts_token_gb300 as moe
from oracle import route_ref as ref

pytestmark = pytest.mark.gpu

SCORES = {True: moe.MOE_SCORE_SIGMOID, False: moe.MOE_SCORE_SOFTMAX}


def call(x, bias, k, sigmoid, groups, top_groups, group_top, renorm, scale,
         **kw):
    T, E = x.shape
    cfg = moe.make_config(T, 8, E, k, 0, 1)
    opt = moe.make_route_scores(SCORES[sigmoid], groups, top_groups,
                                group_top, renorm, scale)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_route_scores(cfg, opt, x.cuda(),
                         None if bias is None else bias.cuda(), idx, w,
                         status, **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy(), status.item()


def check(x, bias, *opt, status=0):
    idx, w, st = call(x, bias, *opt)
    want, ww = ref.route(x.numpy(), None if bias is None else bias.numpy(),
                         *opt)
    assert st == status
    assert np.array_equal(idx, want), np.argwhere((idx != want).any(1))[:4]
    assert np.all(np.abs(w - ww) <= 1e-6 * np.abs(ww) + 1e-37), \
        np.abs(w - ww).max()


# T, E, k, groups, top_groups, group_top: groups of whole lanes and not,
# experts that end inside a lane, one expert, one group of one, all kept
SHAPES = [(1, 256, 8, 8, 4, 2), (77, 256, 8, 8, 4, 2), (33, 1, 1, 1, 1, 1),
          (9, 2, 1, 2, 1, 1),
          (40, 60, 4, 1, 1, 1), (40, 60, 5, 4, 2, 2), (12, 60, 12, 5, 3, 4),
          (65, 128, 6, 4, 2, 1), (19, 160, 6, 8, 3, 1), (31, 95, 16, 1, 1, 1),
          (21, 512, 8, 8, 1, 2), (13, 1024, 32, 64, 9, 3),
          (11, 1000, 20, 4, 4, 2), (17, 32, 32, 1, 1, 1), (8, 64, 8, 64, 8, 1),
          (15, 400, 16, 2, 1, 2), (15, 96, 3, 3, 2, 4), (10, 7, 7, 7, 7, 1)]


@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", SHAPES)
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_random(T, E, k, groups, top_groups, group_top, sigmoid, with_bias,
                renorm):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, E, generator=g) * 2
    bias = torch.randn(E, generator=g) * 0.05 if with_bias else None
    check(x, bias, k, sigmoid, groups, top_groups, group_top, renorm, 2.5)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 4), (6, 2)])
def test_equal_scores_go_to_the_lower_index(sigmoid, groups, top_groups):
    """Few distinct values, and rows of one value only."""
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-2, 3, (50, 192), generator=g).float()
    x[7:12] = 0.0
    x[12, ::2] = -0.0
    x[13:15] = torch.finfo(torch.float32).min
    bias = torch.randint(0, 2, (192,), generator=g).float() * 0.25
    for b in (None, bias, torch.zeros(192)):
        check(x, b, 8, sigmoid, groups, top_groups, 2, True, 1.0)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_near_ties_rank_as_in_64_bits(sigmoid):
    """Scores that float32 cannot tell apart: neighbouring logits, and a bias
    that makes up for a logit to within 2^-24."""
    g = torch.Generator().manual_seed(2)
    T, E = 200, 128
    x = torch.randn(T, E, generator=g)
    near = x[:, :1].expand(T, 16).clone()
    for j in range(16):       # 0..3 ulps from each other, in any order
        for _ in range(j % 4):
            near[:, j] = torch.nextafter(near[:, j], torch.tensor(9.0))
    x[:, 40:56] = near + 1.5
    x[:, 90:106] = near + 1.5
    check(x, None, 20, sigmoid, 1, 1, 1, True, 1.0)
    check(x, torch.zeros(E), 20, sigmoid, 8, 5, 2, True, 1.0)
    s = np.stack([ref.scores(r.astype(np.float64), sigmoid)
                  for r in x.numpy()[:1]])[0]
    bias = torch.from_numpy((s.max() - s).astype(np.float32))
    check(x[:1], bias, 12, sigmoid, 4, 2, 2, False, 1.0)


@pytest.mark.parametrize("E", [100, 128, 200, 256, 500, 1000, 1024])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("ulps", [0, 1])
@pytest.mark.parametrize("shift", [0.0, -8.0])
def test_neighbours_that_are_equal_at_the_last_place(E, sigmoid, with_bias,
                                                     ulps, shift):
    """Of the experts that one lane has, two are far ahead and two or more, equal
    or an ulp apart, share the third place, which is the last one chosen."""
    g = torch.Generator().manual_seed(19)
    per = 2 ** (-(-E // 32) - 1).bit_length()            # experts of a lane
    bias = torch.full((E,), 0.125) if with_bias else None
    for more in (0, 1, 4):           # chosen in other lanes
        x = torch.randn(64, E, generator=g) * 0.5 + shift
        for t in range(64):
            at = torch.randint(0, E // per, (1,), generator=g).item() * per
            mine = at + torch.randperm(per, generator=g)[:4 + t % 3]
            top = torch.tensor(shift + 3 + torch.rand(1, generator=g).item())
            x[t, mine] = top
            x[t, mine[0]], x[t, mine[1]] = top + 2, top + 1
            if ulps:
                x[t, mine[2]] = torch.nextafter(top, torch.tensor(9.0))
            far = torch.randperm(E, generator=g)
            far = far[(far < at) | (far >= at + per)][:more]
            x[t, far] = top + 0.5 + torch.arange(more) * 0.1
        check(x, bias, 3 + more, sigmoid, 1, 1, 1, True, 1.0)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_far_logits(sigmoid):
    """All scores tiny or all saturated, and rows that span float32."""
    x = torch.linspace(-300, 300, 64).repeat(6, 1)
    x[1] = -80 - torch.arange(64.0)
    x[2] = -1000 + torch.arange(64.0)
    x[3] = 60 + torch.arange(64.0) % 7
    x[4] = torch.finfo(torch.float32).min
    x[4, 9] = torch.finfo(torch.float32).max
    x[5] = torch.linspace(-3e38, 3e38, 64)
    # (the last row's steps overflow on some hosts: it may hold NaN)
    status = 0 if x.isfinite().all() else moe.MOE_DEV_NONFINITE
    check(x, None, 5, sigmoid, 1, 1, 1, True, 1.0, status=status)


def test_sigmoid_over_its_range():
    """The weight of one expert is the sigmoid of its logit: the exponential
    and the reciprocal within an ulp (2^-23), a sum and a product rounded
    (2^-24 each)."""
    g = torch.Generator().manual_seed(16)
    x = torch.cat([torch.linspace(-79.99, 40, 150_001),
                   torch.randn(20_000, generator=g) * 3,
                   torch.logspace(-30, 38, 2000), -torch.logspace(-30, 1.9,
                                                                  2000)])
    idx, w, st = call(x[:, None].contiguous(), None, 1, True, 1, 1, 1, False,
                      1.0)
    v = x.double().numpy()
    want = np.exp(np.minimum(v, 0)) / (1 + np.exp(-np.abs(v)))
    assert st == 0 and not idx.any()
    assert np.all(np.abs(w[:, 0] - want) <= 3 * 2.0 ** -23 * want)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scale", [1.0, 1e30, -3e38])
@pytest.mark.parametrize("with_bias", [True, False])
def test_scores_below_float32_beside_others(sigmoid, renorm, scale,
                                            with_bias):
    """Chosen scores of which some are too small for float32 and others are
    not, also under a scale that brings them back: each weight to 1e-6 of
    itself.  Logits are multiples of an eighth, whose differences are exact;
    2^-149 is the smallest step of the result."""
    x = torch.tensor([
        [-59, -70, -100, -130, -200, -1000],
        [-59.125, -59.25, -87.5, -87.625, -95, -103],
        [-0.5, -86.5, -87.5, -88.5, -104.5, -110],
        [200, 120, 113, 96, 90, 5], [-100] * 6,
        [-79.875, -80, -80.125, -80.25, -81, -82],
        [3e38, 0, -1, -100, -1e30, -3e38], [0, -1, -2, -3, -4, -5]])
    x = torch.cat([x, torch.full((len(x), 10), -2000.0)], 1)
    x[6, 6:] = -3.2e38
    bias = torch.zeros(16) if with_bias else None
    opt = (6, sigmoid, 1, 1, 1, renorm, scale)
    idx, w, st = call(x, bias, *opt)
    want, ww = ref.route(x.numpy(), None if bias is None else bias.numpy(),
                         *opt)
    assert st == 0 and np.array_equal(idx, want)
    assert np.all(np.abs(w - ww) <= 1e-6 * np.abs(ww) + 2.0 ** -149), \
        np.argwhere(np.abs(w - ww) > 1e-6 * np.abs(ww))


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 2),
                                                         (3, 1, 1)])
def test_nonfinite_logits_and_bias(sigmoid, groups, top_groups, group_top):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(20, 48, generator=g)
    x[0] = float("nan")
    x[1, 5], x[2, 6], x[3, 7] = float("nan"), float("inf"), float("-inf")
    x[4, :46] = float("-inf")
    x[5, 16:] = float("inf")
    opt = (6, sigmoid, groups, top_groups, group_top, True, 1.0)
    check(x, None, *opt, status=moe.MOE_DEV_NONFINITE)
    check(x[6:], None, *opt)
    bias = torch.randn(48, generator=g) * 0.1
    check(x, bias, *opt, status=moe.MOE_DEV_NONFINITE)
    bias[9], bias[20] = float("nan"), float("inf")
    check(x[6:], bias, *opt, status=moe.MOE_DEV_NONFINITE)


def test_large_bias_leaves_no_choice_to_rounding():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(30, 64, generator=g)
    bias = torch.full((64,), 1e6)
    check(x, bias, 8, True, 4, 2, 2, True, 1.0)
    bias = torch.randn(64, generator=g) * 1e30
    check(x, bias, 8, False, 4, 2, 2, True, 1.0)


@pytest.mark.parametrize("E,groups,top_groups,group_top",
                         [(256, 1, 1, 1), (256, 8, 4, 1), (60, 1, 1, 1),
                          (60, 4, 2, 2), (1000, 1, 1, 1), (28, 1, 1, 1)])
@pytest.mark.parametrize("score,shift", [("logit", 0.0), ("sigmoid", -0.5),
                                         ("softmax", -1.0)])
def test_zeros_and_subnormals_between_other_rows(E, groups, top_groups,
                                                 group_top, score, shift):
    """c of zero, of both signs, below the smallest normal number, as low as
    numbers go and beyond, in rows that one warp has one after another."""
    g = torch.Generator().manual_seed(14)
    kinds = [torch.randn(E, generator=g), torch.zeros(E),
             torch.arange(E) * 1e-44, -torch.arange(E) * 1e-42,
             torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0),
             torch.full((E,), -3.4028234e38), torch.full((E,), -3.4e38),
             3e38 - torch.arange(E) * 1e36 * (600 / E)]
    x = torch.stack(kinds * 40).float()
    x = x.repeat(16, 1)
    bias = None if score == "logit" else torch.full((E,), shift)
    opt = (6, score != "softmax", groups, top_groups, group_top, False, 1.0)
    idx, w, st = call(x, bias, *opt)
    want, ww = ref.route(x[:len(kinds)].numpy(),
                         None if bias is None else bias.numpy(), *opt)
    # the last kind ends in infinities
    assert not torch.isfinite(kinds[-1]).all()
    assert st == moe.MOE_DEV_NONFINITE
    assert np.array_equal(idx, np.tile(want, (40 * 16, 1)))
    ww = np.tile(ww, (40 * 16, 1))
    assert np.all(np.abs(w - ww) <= 1e-6 * np.abs(ww) + 1e-37)


# E, groups, group_top: groups of whole lanes that end before the warp does,
# with one to sixteen experts a lane
@pytest.mark.parametrize("E,groups,group_top", [
    (16, 8, 1), (24, 3, 2), (28, 7, 1), (48, 3, 2), (48, 6, 1), (96, 3, 2),
    (112, 7, 2), (160, 5, 2), (192, 6, 1), (240, 15, 2), (448, 7, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_near_groups_that_leave_lanes_empty(E, groups, group_top, sigmoid,
                                            with_bias):
    """Equal and nearly equal group sums: what is looked at more closely ends
    with the last expert, of the last token and of the bias too."""
    g = torch.Generator().manual_seed(15)
    size = E // groups
    x = torch.randn(24, E, generator=g)
    x[:8] = x[:8, :size].repeat(1, groups)          # equal sums
    x[8:16] = x[8:16, :size].repeat(1, groups)      # sums an ulp apart
    odd = x[8:16, size::2 * size]                   # every other group's first
    x[8:16, size::2 * size] = torch.nextafter(odd, torch.tensor(9.0))
    x[16] = 0.0
    bias = torch.full((E,), 0.25) if with_bias else None
    for top_groups in {1, groups - 1}:
        k = min(top_groups * size, 4)
        opt = (k, sigmoid, groups, top_groups, group_top, True, 1.0)
        check(x, bias, *opt)
        check(x[15:16].clone(), bias, *opt)         # a single token


def test_unaligned_logits_and_other_stream():
    g = torch.Generator().manual_seed(5)
    flat = torch.randn(33 * 128 + 1, generator=g).cuda()
    x = flat[1:].view(33, 128)
    assert x.data_ptr() % 16 == 4
    opt = (8, True, 4, 2, 2, True, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    idx, w, _ = call(x, None, *opt, stream=side)
    want, ww = ref.route(x.cpu().numpy(), None, *opt)
    assert np.array_equal(idx, want) and np.allclose(w, ww, rtol=1e-6)


def test_more_tokens_than_warps_of_a_grid():
    g = torch.Generator().manual_seed(6)
    T, E = 140_000, 8
    x = torch.randn(T, E, generator=g)
    idx, w, _ = call(x, None, 2, False, 1, 1, 1, False, 1.0)
    want = np.argsort(-x.numpy(), 1, kind="stable")[:, :2]
    assert np.array_equal(idx, want)
    p = x.double().softmax(1).numpy()
    assert np.allclose(w, np.take_along_axis(p, want, 1), rtol=1e-6)


def test_no_tokens():
    cfg = moe.make_config(0, 8, 16, 2, 0, 1)
    opt = moe.make_route_scores(groups=4, top_groups=2)
    moe.moe_route_scores(cfg, opt, None, None, None, None)
    moe.moe_route_scores_backward(cfg, opt, None, None, None, None)


# ---------------------------------------------------------- backward -----
def back(x, idx, dw, sigmoid, renorm, scale):
    T, E = x.shape
    cfg = moe.make_config(T, 8, E, idx.shape[1], 0, 1)
    opt = moe.make_route_scores(SCORES[sigmoid], renorm=renorm, scale=scale)
    out = torch.full((T, E), 7.0, device="cuda")
    moe.moe_route_scores_backward(cfg, opt, x.cuda(),
                                  idx.int().cuda(), dw.cuda(), out)
    torch.cuda.synchronize()
    return out.cpu().numpy()


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (33, 256, 8), (9, 1, 1),
                                   (40, 60, 4), (7, 95, 16), (5, 1024, 32),
                                   (11, 1000, 20), (6, 3, 3)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward(T, E, k, sigmoid, renorm):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, E, generator=g) * 2
    dw = torch.randn(T, k, generator=g)
    idx = torch.rand(T, E, generator=g).topk(k).indices
    got = back(x, idx, dw, sigmoid, renorm, 2.5)
    want = ref.route_backward(x.numpy(), idx.numpy(), dw.double().numpy(),
                              sigmoid, renorm, 2.5)
    s = np.stack([ref.scores(r.astype(np.float64), sigmoid)
                  for r in x.numpy()])
    ch = np.take_along_axis(s, idx.numpy(), 1)
    terms = 2.5 * np.abs(dw.numpy()).sum(1, keepdims=True) * (
        1 / ch.sum(1, keepdims=True) if renorm else 1)
    tol = 2e-6 * terms * s + 1e-37
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("sigmoid", [True, False])
def test_backward_unaligned_nonfinite_and_odd_indexes(sigmoid):
    g = torch.Generator().manual_seed(8)
    E, k = 128, 4
    x = torch.randn(6, E, generator=g)
    idx = torch.rand(6, E, generator=g).topk(k).indices
    dw = torch.randn(6, k, generator=g)
    clean = back(x, idx, dw, sigmoid, True, 1.0)
    flat = torch.zeros(6 * E + 3).cuda()
    flat[3:] = x.reshape(-1)
    assert np.allclose(back(flat[3:].view(6, E), idx, dw, sigmoid, True, 1.0),
                       clean, rtol=1e-5, atol=1e-9)
    # a chosen logit that is not finite, an index outside, one that is twice
    x[1, idx[1, 0]] = float("nan")
    x[2, idx[2, 1]] = float("inf")
    out = idx.clone()
    out[3, 2], out[4, 0] = -1, E
    out[5, 1] = out[5, 0]
    got = back(x, out, dw, sigmoid, False, 1.0)
    assert np.isfinite(got).all()
    assert got[1, idx[1, 0]] == 0 and got[2, idx[2, 1]] == 0
    xs = torch.where(x.isfinite(), x, torch.tensor(float("-inf"))).numpy()
    for t in range(6):
        keep = [j for j in range(k) if 0 <= out[t, j] < E
                and np.isfinite(x[t, out[t, j]])]
        want = ref.route_backward(xs[t:t + 1], out[t:t + 1, keep].numpy(),
                                  dw[t:t + 1, keep].double().numpy(), sigmoid,
                                  False, 1.0)
        assert np.allclose(got[t], want[0], rtol=1e-5, atol=1e-7), t


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scale", [1.0, 1e30, -3e38])
@pytest.mark.parametrize("E", [16, 19])
def test_backward_of_scores_below_float32_beside_others(sigmoid, renorm,
                                                        scale, E):
    """Scores, and what they lack of 1, that are too small for float32 without
    the scale: test_backward's bound of each entry by its own score (and by
    1 - s), with the smallest step of the result.  Logits are multiples of an
    eighth, whose differences are exact."""
    x = torch.tensor([
        [-59, -70, -100, -130, -150, -1000],
        [-59.125, -59.25, -87.5, -87.625, -95, -103],
        [-0.5, -86.5, -87.5, -88.5, -104.5, -110],
        [100, 89, 88.5, 95, 81, 5], [-100] * 6, [140, 130, 100, 90, 85, 81],
        [-79.875, -80, -80.125, -80.25, -81, -82], [0, -1, -2, -3, -4, -5]])
    g = torch.Generator().manual_seed(17)
    x = torch.cat([x, torch.randint(-160, 0, (len(x), E - 6), generator=g)
                   + x[:, :1]], 1)
    dw = (torch.rand(len(x), 6, generator=g) - 0.5) * 0.1
    idx = torch.arange(6).repeat(len(x), 1)
    idx[:, 3] = E - 2                                # one of the others
    got = back(x, idx, dw, sigmoid, renorm, scale)
    want = ref.route_backward(x.numpy(), idx.numpy(), dw.double().numpy(),
                              sigmoid, renorm, scale)
    x64 = x.double().numpy()
    s = np.exp(np.stack([ref.log_scores(r, sigmoid) for r in x64]))
    ch = np.take_along_axis(s, idx.numpy(), 1)
    terms = abs(scale) * np.abs(dw.double().numpy())
    terms = terms.max(1, keepdims=True) * 2 / ch.sum(1, keepdims=True) \
        if renorm else terms.max(1, keepdims=True) if sigmoid else \
        (terms * ch).sum(1, keepdims=True) + terms.max(1, keepdims=True)
    tol = 4e-6 * terms * s + 2.0 ** -149
    if sigmoid:
        tol = 4e-6 * terms * s / (1 + np.exp(x64)) + 2.0 ** -149
    assert np.all(np.abs(got - want) <= tol), \
        np.argwhere(np.abs(got - want) > tol)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("k", [2, 6, 13, 20])
def test_a_token_is_routed_alike_beside_any_others(sigmoid, renorm, k):
    """Rows with far scores, NaN or ties between them change no bit of others:
    neither of the weights nor of the gradient."""
    g = torch.Generator().manual_seed(20)
    T, E = 61, 96
    x = torch.randn(T, E, generator=g) * 2
    dw = torch.randn(T, k, generator=g)
    opt = (k, sigmoid, 6, 4, 2, renorm, 2.5)
    idx, w, _ = call(x, None, *opt)
    dl = back(x, torch.from_numpy(idx), dw, sigmoid, renorm, 2.5)
    other = x.clone()
    other[1::4] = x[1::4] * 60 - 200
    other[2::8, 5] = float("nan")
    other[6::8] = 1.0
    keep = np.ones(T, dtype=bool)
    keep[1::4] = keep[2::8] = keep[6::8] = False
    i2, w2, _ = call(other, None, *opt)
    d2 = back(other, torch.from_numpy(i2), dw, sigmoid, renorm, 2.5)
    assert np.array_equal(idx[keep], i2[keep])
    assert np.array_equal(w[keep], w2[keep])
    assert np.array_equal(dl[keep], d2[keep])


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_beside_a_bias_that_is_not_finite(sigmoid, renorm):
    """Experts chosen for want of others, whose weight is 0: with their indexes
    taken out the gradient is that of the weights."""
    g = torch.Generator().manual_seed(18)
    T, E, k = 9, 12, 5
    x = torch.randn(T, E, generator=g)
    bias = torch.randn(E, generator=g) * 0.1
    bias[3:] = torch.tensor([float("nan"), float("inf"), float("-inf")] * 3)
    opt = (k, sigmoid, 1, 1, 1, renorm, 2.5)
    idx, w, st = call(x, bias, *opt)
    want, ww = ref.route(x.numpy(), bias.numpy(), *opt)
    assert st == moe.MOE_DEV_NONFINITE and np.array_equal(idx, want)
    lost = idx >= 3
    assert (lost.sum(1) == 2).all() and not w[lost].any()
    dw = torch.randn(T, k, generator=g)
    got = back(x, torch.from_numpy(np.where(lost, -1, idx)), dw, sigmoid,
               renorm, 2.5)
    dl = ref.route_backward(x.numpy(), idx[:, :3], dw[:, :3].double().numpy(),
                            sigmoid, renorm, 2.5)
    assert np.allclose(got, dl, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_forward_and_backward_in_a_graph(sigmoid):
    """Captured once, replayed on other logits."""
    g = torch.Generator().manual_seed(9)
    T, E, k = 37, 256, 8
    cfg = moe.make_config(T, 8, E, k, 0, 1)
    opt = moe.make_route_scores(SCORES[sigmoid], 8, 4, 2, True, 2.5)
    x, bias = torch.zeros(T, E).cuda(), (torch.randn(E, generator=g)
                                         * 0.05).cuda()
    dw = torch.randn(T, k, generator=g).cuda()
    idx = torch.zeros(T, k, dtype=torch.int32).cuda()
    w, dl = torch.zeros(T, k).cuda(), torch.zeros(T, E).cuda()

    def step():
        moe.moe_route_scores(cfg, opt, x, bias, idx, w)
        moe.moe_route_scores_backward(cfg, opt, x, idx, dw, dl)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        new = torch.randn(T, E, generator=g)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want, ww = ref.route(new.numpy(), bias.cpu().numpy(), k, sigmoid, 8,
                             4, 2, True, 2.5)
        assert np.array_equal(idx.cpu().numpy(), want)
        wd = ref.route_backward(new.numpy(), want, dw.cpu().double().numpy(),
                                sigmoid, True, 2.5)
        assert np.allclose(dl.cpu().numpy(), wd, rtol=1e-4, atol=1e-6)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_two_calls_at_once(sigmoid):
    """Calls on two streams that overlap, each with memory of its own."""
    g = torch.Generator().manual_seed(12)
    T, E, k = 3000, 256, 8
    cfg = moe.make_config(T, 8, E, k, 0, 1)
    opt = moe.make_route_scores(SCORES[sigmoid], 8, 4, 2, True, 2.5)
    bias = (torch.randn(E, generator=g) * 0.05).cuda()
    dw = torch.randn(T, k, generator=g).cuda()
    xs = [torch.randn(T, E, generator=g).cuda() for _ in range(2)]
    outs = [(torch.zeros(T, k, dtype=torch.int32).cuda(),
             torch.zeros(T, k).cuda(), torch.zeros(T, E).cuda())
            for _ in range(4)]

    def step(x, o, **kw):
        moe.moe_route_scores(cfg, opt, x, bias, o[0], o[1], **kw)
        moe.moe_route_scores_backward(cfg, opt, x, o[0], dw, o[2], **kw)
    for x, o in zip(xs, outs):
        step(x, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, o, s in zip(xs, outs[2:], streams):
            step(x, o, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(outs[:2], outs[2:]):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_inputs_written_by_the_kernel_before():
    """Logits that change between calls, by torch and by the backward."""
    g = torch.Generator().manual_seed(13)
    T, E, k = 2000, 64, 6
    cfg = moe.make_config(T, 8, E, k, 0, 1)
    opt = moe.make_route_scores(moe.MOE_SCORE_SOFTMAX, 1, 1, 1, False, 1.0)
    src = [torch.randn(T, E, generator=g).cuda() for _ in range(4)]
    x, dl = torch.zeros(T, E).cuda(), torch.zeros(T, E).cuda()
    dw = torch.ones(T, k).cuda()
    idx = [torch.zeros(T, k, dtype=torch.int32).cuda() for _ in range(8)]
    w = torch.zeros(T, k).cuda()
    grads = []
    for i in range(4):
        x.copy_(src[i])
        moe.moe_route_scores(cfg, opt, x, None, idx[i], w)
        moe.moe_route_scores_backward(cfg, opt, x, idx[i], dw, dl)
        moe.moe_route_scores(cfg, opt, dl, None, idx[4 + i], w)
        grads.append(dl.clone())
    torch.cuda.synchronize()
    for got, rows in zip(idx, src + grads):
        want = np.argsort(-rows.cpu().numpy(), 1, kind="stable")[:, :k]
        assert np.array_equal(got.cpu().numpy(), want)

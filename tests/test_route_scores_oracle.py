"""The oracle of routing by scores against small cases by hand, and its
gradient against differences (CPU)."""
import numpy as np
import pytest

from oracle import route_ref as ref


def test_groups_bias_and_ties_by_hand():
    # sigmoid(0) = 1/2 everywhere: the bias alone ranks
    x = np.zeros((1, 6), dtype=np.float32)
    b = np.array([0.3, 0.0, 0.2, 0.2, 0.1, 0.1], dtype=np.float32)
    idx, w = ref.route(x, b, 3, True, 3, 2, 2, True, 2.5)
    # group sums .3 .4 .2 (and 1 each): groups 1 and 0
    assert idx.tolist() == [[0, 2, 3]]
    assert np.allclose(w, 2.5 / 3)
    idx, _ = ref.route(x, b, 2, True, 3, 1, 1, False, 1.0)
    assert idx.tolist() == [[0, 1]]       # the largest: group 0
    idx, _ = ref.route(x, None, 4, False, 1, 1, 1, False, 1.0)
    assert idx.tolist() == [[0, 1, 2, 3]]


def test_nonfinite_experts_rank_last():
    x = np.array([[np.nan, 1.0, np.inf, -3.0]], dtype=np.float32)
    idx, w = ref.route(x, None, 4, True, 1, 1, 1, False, 1.0)
    assert idx.tolist() == [[1, 3, 0, 2]]
    assert w[0, 2] == w[0, 3] == 0


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(sigmoid, renorm):
    g = np.random.default_rng(0)
    x = g.normal(size=(1, 9))
    idx = np.array([[4, 0, 7]])
    dw = g.normal(size=(1, 3))

    def loss(v):
        s = ref.scores(v[0], sigmoid)[idx[0]]
        return 1.7 * (dw[0] * (s / s.sum() if renorm else s)).sum()
    got = ref.route_backward(x, idx, dw, sigmoid, renorm, 1.7)
    for e in range(9):
        h = np.zeros((1, 9))
        h[0, e] = 1e-5
        d = (loss(x + h) - loss(x - h)) / 2e-5
        assert abs(d - got[0, e]) < 1e-8, e

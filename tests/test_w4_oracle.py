"""The 4-bit oracle against a loop over single weights (CPU)."""
import numpy as np
import pytest

from oracle import w4_ref as ref


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_dequantize_is_the_formula(group, zeros):
    g = np.random.default_rng(0)
    n, K, N = 2, 72, 3
    G = -(-K // group)
    codes = g.integers(0, 256, (n, K // 2, N), dtype=np.uint8)
    scales = g.normal(size=(n, G, N))
    zp = g.integers(0, 16, (n, G, N), dtype=np.uint8) if zeros else None
    got = ref.dequantize(codes, scales, zp, group)
    for m in range(n):
        for k in range(K):
            for c in range(N):
                q = (int(codes[m, k // 2, c]) >> (4 * (k % 2))) & 15
                z = int(zp[m, k // group, c]) if zeros else 8
                assert got[m, k, c] == (q - z) * scales[m, k // group, c]


def test_swiglu_groups_and_map():
    g = np.random.default_rng(1)
    wg, wu, wd = (g.normal(size=s) for s in ((2, 4, 6), (2, 4, 6), (2, 6, 4)))
    x = g.normal(size=(5, 4))
    h, y = ref.swiglu(x, [0, 2, 2, 5], [1, 0, 1], wg, wu, wd)
    a, b = x @ wg[1], x @ wu[1]
    assert np.allclose(h, a / (1 + np.exp(-a)) * b)
    assert np.allclose(y, h @ wd[1])

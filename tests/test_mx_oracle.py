"""The oracle of microscaled 4-bit numbers against cases by hand (CPU)."""
import numpy as np

from oracle import mx_ref as ref


def test_codes_are_the_nearest_and_ties_go_to_the_even_code():
    # the largest, 6, makes the scale 1 in either form
    x = np.zeros((1, 32))
    x[0, :10] = [6, 0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, -0.26, 0.24]
    want = [6, 0, 1, 1, -2, 2, 4, 4, -0.5, 0]
    for block, one in ((32, 127), (16, 0x38)):
        codes, scales = ref.quantize_rows(x, block)
        assert scales[0, 0] == one
        assert ref.dequantize_rows(codes, scales, block)[0, :10].tolist() == \
            want


def test_scales_by_hand():
    x = np.zeros((1, 128))
    x[0, 0], x[0, 32], x[0, 96] = 7.9, -0.124, np.inf
    codes, scales = ref.quantize_rows(x, 32)
    assert scales.tolist() == [[127, 121, 0, 255]]   # 2^0, 2^-6, 2^-127, NaN
    v = ref.dequantize_rows(codes, scales, 32)
    assert v[0, 0] == 6 and v[0, 32] == -6 * 2.0 ** -6
    assert np.isnan(v[0, 96:]).all() and not v[0, 64:96].any()
    x = np.zeros((1, 64))
    x[0, 0], x[0, 16], x[0, 32], x[0, 48] = 3000.0, 6.0, 0.005, np.nan
    codes, scales = ref.quantize_rows(x, 16)
    # 448 at most, 1, 0.005 / 6 is below half of 2^-9, NaN
    assert scales.tolist() == [[126, 0x38, 0, 127]]
    v = ref.dequantize_rows(codes, scales, 16)
    assert v[0, 0] == 448 * 6 and v[0, 16] == 6 and v[0, 32] == 0
    assert np.isnan(v[0, 48:]).all()


def test_every_small_float_is_its_own_nearest():
    for b in range(127):
        assert ref.nearest_small(ref.SMALL[b]) == b
    mid = (ref.SMALL[8] + ref.SMALL[9]) / 2
    assert ref.nearest_small(mid) == 8


def test_rows_of_scales_end_in_zeros():
    codes, scales = ref.quantize_rows(np.ones((2, 160)), 32)
    assert codes.shape == (2, 80) and scales.shape == (2, 8)
    assert not scales[:, 5:].any() and scales[:, :5].all()

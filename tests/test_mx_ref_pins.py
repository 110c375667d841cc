"""The plain 64-bit forms of the microscaled operators (tests/mx_ref.py) on
hand-worked values; no GPU."""
import numpy as np
import pytest

import mx_ref as R


def test_tables():
    assert R.E4M3[-1] == 448.0 and R.E4M3[1] == 2.0 ** -9 and R.E4M3[8] == 2.0 ** -6 and len(R.E4M3) == 127


def test_ties_go_to_the_even_code():
    # 0.25 lies between codes 0 and 1, 0.75 between 1 and 2, ... 5 between 6 (4.0) and 7 (6.0)
    got = R.E2M1[R.nearest(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9]), R.E2M1)]
    assert got.tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]


def test_mx4_block():
    x = np.zeros((1, 33))
    x[0, 0], x[0, 1], x[0, 2], x[0, 32] = 7.9, -1.0, 0.3, 3.0
    val, codes, byte = R.mx4(x)
    # amax 7.9: s = 2 - 2 = 0; the second block's amax 3: s = 1 - 2 = -1, 3 / 0.5 = 6
    assert byte.tolist() == [[127, 126]]
    assert val[0, :3].tolist() == [6.0, -1.0, 0.5] and val[0, 32] == 3.0
    packed, scales = R.pack4(codes, byte)
    assert packed.shape == (1, 32) and packed[0, 0] == (7 | (8 + 2) << 4) and packed[0, 1] == 1 and packed[0, 16] == 7
    assert scales[0, 0, 0, 0].tolist() == [127, 126, 0, 0]


def test_act8_scale_is_the_smallest_that_does_not_saturate():
    for a, s in ((448.0, 0), (448.5, 1), (1.75, -8), (1.76, -7), (1.0, -8)):
        val, codes, byte = R.act8(np.array([[a]]))
        assert byte[0, 0] == s + 127 and abs(val[0, 0] - a) <= a / 16


@pytest.mark.parametrize("f", [R.mx4, R.act8])
def test_not_finite_and_zero_blocks(f):
    x = np.zeros((3, 32))
    x[0, 5], x[1, 7] = np.nan, -np.inf
    val, codes, byte = f(x)
    assert byte[:, 0].tolist() == [255, 255, 0]
    assert np.isnan(val[:2]).all() and (val[2] == 0).all() and (codes[:2] == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slope_against_differences(act):
    g = np.linspace(-9, 9, 181)
    d = 1e-5
    diff = (R.gate(act, g + d) - R.gate(act, g - d)) / (2 * d)
    # the central difference is off by d^2 / 6 times the third derivative (below 2) plus 2^-53 * 9 / d
    assert np.max(np.abs(diff - R.gate_slope(act, g))) < d * d + 2.0 ** -52 * 9 / d

"""The microscaled 4-bit reference against hand-worked blocks (CPU)."""
import numpy as np
import pytest

import mxfp4_reference as R


def test_hand_worked_block():
    # max 5 lies in [4, 8): scale 2^0; 5 ties between 4 and 6 and goes to the even code of 4
    x = np.zeros((1, 32))
    x[0, :8] = [5.0, -0.25, 0.75, 0.26, -3.5, 2.5, 1.25, -1.75]
    c, s = R.quantize(x)
    assert s[0].tolist() == [127, 127, 127, 127]
    nib = np.stack((c & 15, c >> 4), -1).reshape(-1)
    assert nib[:8].tolist() == [6, 8 + 0, 2, 1, 8 + 6, 4, 2, 8 + 4]
    assert not nib[8:].any()


@pytest.mark.parametrize("a,scale,largest", [(4.0, 127, 4.0), (7.9, 127, 6.0), (8.0, 128, 8.0), (1.0, 125, 1.0),
                                             (2.0 ** -126, 0, 2.0 ** -126), (2.0 ** -130, 0, 0.0), (3e38, 252, 6 * 2.0 ** 125)])
def test_scale_of_the_largest(a, scale, largest):
    x = np.zeros((1, 3))
    x[0, 1] = -a
    c, s = R.quantize(x)
    assert s[0, 0] == scale
    assert R.values(c, s)[0, 1] == -largest


def test_not_finite_blocks_and_padding():
    x = np.ones((2, 70))
    x[0, 3], x[1, 40] = np.nan, -np.inf
    c, s = R.quantize(x)
    assert s.tolist() == [[255, 125, 125, 127], [125, 255, 125, 127]]
    v = R.values(c, s)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 32:64]).all()
    assert (v[0, 32:70] == 1).all() and not v[:, 70:96].any() and not v[:, 96:].any()


def test_values_are_their_own_quantisation():
    rng = np.random.default_rng(5)
    c, s = R.random_operand(rng, 5, 300)
    v = R.values(c, s)
    c2, s2 = R.quantize(v[:, :300])
    assert (R.values(c2, s2) == v).all()

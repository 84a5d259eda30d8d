"""Pins of the 4-bit oracle: hand-worked roundings, scales at the ends of their range, the stored layout."""
import numpy as np
import pytest

from oracle import mx4


def _block(vals):
    x = np.zeros((1, 32))
    x[0, :len(vals)] = vals
    return x


def test_roundings_by_hand():
    # 6 fixes the scale at 1; ties go to the even code: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    vals = [6, .25, .26, .75, .74, 1.25, 1.75, 2.5, 2.51, 3.5, 3.49, 5, 5.01, -5, -.25, 7.9]
    want = [6, 0, .5, 1, .5, 1, 2, 2, 3, 4, 3, 4, 6, -4, 0, 6]
    code, s = mx4.quantize(_block(vals))
    assert s[0, 0] == 127
    assert np.array_equal(mx4.values(code, s, 16)[0], want)
    assert code[0, 14] == 8  # minus zero keeps its sign


@pytest.mark.parametrize("top,e", [(4.0, 0), (3.999, -1), (7.99, 0), (8.0, 1), (2.0 ** -125, -127), (2.0 ** -126, -127),
                                   (2.0 ** -149, -127), (0.0, -127), (3.4e38, 125)])
def test_scale(top, e):
    _, s = mx4.quantize(_block([top]))
    assert s[0, 0] == e + 127


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_non_finite_block_is_nan_and_only_it(bad):
    x = np.ones((2, 64))
    x[0, 3] = bad
    v = mx4.roundtrip(x)
    assert np.isnan(v[0, :32]).all()
    assert (v[0, 32:] == 1).all() and (v[1] == 1).all()


def test_relative_error_of_a_roundtrip():
    # the largest value lies in [4, 8) scales, the grid's step there is 2, and 8 saturates to 6: off by at most 2 scales
    x = np.random.default_rng(0).standard_normal((50, 320))
    v = mx4.roundtrip(x)
    e = np.floor(np.log2(np.abs(x.reshape(50, 10, 32)).max(-1))) - 2
    assert (np.abs(v - x).reshape(50, 10, 32) <= 2.0 * np.exp2(e)[..., None]).all()


@pytest.mark.parametrize("rows,k", [(1, 1), (63, 31), (65, 129), (130, 300)])
def test_store_and_load(rows, k):
    code, s = mx4.quantize(np.random.default_rng(rows).standard_normal((rows, k)))
    codes, tiles = mx4.store(code, s)
    assert codes.shape == (rows, -(-k // 128) * 64) and tiles.shape == (-(-rows // 64), -(-k // 128), 64, 4)
    c2, s2 = mx4.load(codes, tiles)
    assert np.array_equal(code, c2) and np.array_equal(s, s2)
    assert (code[:, k:] == 0).all()

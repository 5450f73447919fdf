"""Pins of the row-scaled and grouped oracle: exact rational arithmetic, hand
values, and the sum over groups against the dense oracle."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import fp8_oracle as O
from oracle import rows_oracle as R


def test_i8_scale_hand_values():
    assert R.i8_row_scale(127.0) == 1.0
    assert R.i8_row_scale(254.0) == 0.5
    assert R.i8_row_scale(0.0) == 1.0
    assert R.i8_row_scale(np.float32(1e-37)) == 1.0  # 127 / 1e-37 overflows
    assert np.isnan(R.i8_row_scale(np.inf)) and np.isnan(R.i8_row_scale(np.nan))


def test_i8_rounding_ties_to_even():
    q, s = R.i8_quantize_rows(np.float32([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5]]))
    assert s[0] == 1.0
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, 126]


def test_i8_codes_are_the_nearest_integers_of_the_rounded_product():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((8, 33)) * 10.0 ** rng.uniform(-30, 30, (8, 1))).astype(np.float32)
    q, s = R.i8_quantize_rows(x)
    for r in range(8):
        for k in range(33):
            exact = Fraction(float(x[r, k])) * Fraction(float(s[r]))
            v = Fraction(float(np.float32(float(x[r, k]) * float(s[r]))))
            assert abs(v - exact) <= abs(exact) * Fraction(1, 2 ** 24)
            assert abs(Fraction(int(q[r, k])) - v) <= Fraction(1, 2)
    assert np.abs(q.astype(int)).max() == 127 and q.min() >= -127


def test_i8_nonfinite_row_is_marked_and_alone():
    x = np.ones((3, 4), np.float32)
    x[1, 2] = np.nan
    q, s = R.i8_quantize_rows(x)
    assert np.isnan(s[1]) and not q[1].any()
    assert (q[[0, 2]] == 127).all() and (s[[0, 2]] == 127).all()


def test_i8_linear_in_rationals():
    rng = np.random.default_rng(4)
    q = rng.integers(-127, 128, (3, 17)).astype(np.int8)
    w = rng.integers(-127, 128, (5, 17)).astype(np.int8)
    sx, sw = np.float32([2, 0.5, 4]), np.float32([1, 2, 4, 8, 0.25])
    b = np.array([1.0, -2.0, 0.5, 0.0, 3.0])
    r, p = R.i8_linear(q, sx, w, sw, b)
    for m in range(3):
        for n in range(5):
            v = Fraction(sum(int(a) * int(c) for a, c in zip(q[m], w[n]))) / (
                Fraction(float(sx[m])) * Fraction(float(sw[n])))
            assert Fraction(p[m, n]) == v and Fraction(r[m, n]) == v + Fraction(b[n])


@pytest.mark.parametrize("offsets", [[0, 3, 3, 8], [2, 2, 7, 8]])
def test_groups_cover_their_rows_with_their_weights(offsets):
    rng = np.random.default_rng(5)
    x8 = rng.integers(0, 120, (8, 16)).astype(np.uint8)
    w8 = rng.integers(0, 120, (3, 6, 16)).astype(np.uint8)
    sw = np.float32([1, 2, 4])
    refs = R.grouped_fwd(x8, w8, O.E4M3, np.float32(1), sw, offsets)
    for t in range(8):
        owner = [e for e, i, j in R.spans(offsets) if i <= t < j]
        if not owner:
            continue
        e, i, _ = R.spans(offsets)[owner[0]]
        want = (O.decode_array(x8[t], O.E4M3) @ O.decode_array(w8[e], O.E4M3).T) / sw[e]
        np.testing.assert_allclose(refs[e].r[t - i], want, rtol=1e-12)
    dws = R.grouped_dw(x8, O.E4M3, x8, O.E4M3, np.float32(1), np.float32(1), offsets)
    inside = x8[offsets[0]:offsets[-1]]
    total = sum(d.r for d in dws if d is not None)
    dense = O.linear_bwd_dw(inside, O.E4M3, inside, O.E4M3, np.float32(1), np.float32(1)).r
    np.testing.assert_allclose(total, dense, rtol=1e-12)

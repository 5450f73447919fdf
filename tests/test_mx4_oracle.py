"""Pins of the 4-bit floating point oracle: the formats' tables, hand values,
brute force over neighbours."""

import numpy as np
import pytest

from oracle import mx4_oracle as X


def test_elements_are_the_formats():
    assert [X.element(c) for c in range(8)] == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert [X.element(c) for c in range(8, 16)] == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert X.GRID.tolist() == [X.element(c) for c in range(8)]


def test_midpoints_go_to_the_even_code():
    for c in range(7):
        mid = (X.GRID[c] + X.GRID[c + 1]) / 2
        assert X.nearest(mid) == c + c % 2
        assert X.nearest(np.nextafter(mid, 0)) == c and X.nearest(np.nextafter(mid, 9)) == c + 1
    assert X.nearest(7.99) == 7 and X.nearest(0.0) == 0


@pytest.mark.parametrize("amax,e", [(6.0, 127), (4.0, 127), (7.99, 127), (8.0, 128), (3.99, 126),
                                    (1.0, 125), (0.0, 0), (2.0 ** -125, 0), (2.0 ** -149, 0),
                                    (2.0 ** -124, 1), (np.finfo(np.float32).max, 252),
                                    (np.inf, 255), (np.nan, 255)])
def test_exponents(amax, e):
    assert X.exponent(amax) == e


def test_quantize_by_hand():
    x = np.zeros((1, 40))
    x[0, :5] = [6.0, -0.25, 0.75, -5.0, 0.3]
    x[0, 32:34] = [0.01, -0.004]
    c, e = X.quantize(x)
    assert e.tolist() == [[127, 118]]  # 0.01 = 1.28 2^-7: scale 2^-9
    assert c[0, 0, :5].tolist() == [7, 8, 2, 14, 1]
    v = X.values(c, e)
    assert v[0, :5].tolist() == [6, 0, 1, -4, 0.5] and v[0, 32] == 6 / 512 and v[0, 33] == -2 / 512
    x[0, 3] = np.nan
    c, e = X.quantize(x)
    assert e[0, 0] == 255 and not c[0, 0].any() and e[0, 1] == 118
    assert np.isnan(X.values(c, e)[0, :32]).all()


def test_packing():
    c, e = X.quantize(np.arange(2 * 160, dtype=np.float64).reshape(2, 160))
    p, s = X.pack(c, e)
    assert p.shape == (2, 80) and s.shape == (2, 2, 4)
    assert p[1, 3] == c[1, 0, 6] | c[1, 0, 7] << 4
    assert s[0, 1].tolist() == e[1, :4].tolist() and s[1, 0].tolist() == [e[0, 4], 0, 0, 0]


def test_linear_against_a_loop():
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((3, 7)), rng.standard_normal((2, 7)), [1.0, -2.0]
    r, m = X.linear(x, w, b)
    for i in range(3):
        for j in range(2):
            assert r[i, j] == pytest.approx(sum(x[i, k] * w[j, k] for k in range(7)) + b[j])
            assert m[i, j] == pytest.approx(sum(abs(x[i, k] * w[j, k]) for k in range(7)))

"""Pins of the routing oracle: hand values, differences, brute force."""

import numpy as np
import pytest

from oracle import route_oracle as R


def test_choice_by_hand():
    z = [1.0, 3.0, 2.0, 3.0]
    assert R.choose(z, None, R.SOFTMAX, 3) == [1, 3, 2]
    assert R.choose(z, [0, 0, 5.0, 0], R.SIGMOID, 2) == [2, 1]
    assert R.choose(z, [0, -np.inf, 0, 0], R.SIGMOID, 4) == [3, 2, 0, -1]
    assert R.choose([-np.inf] * 3, None, R.SOFTMAX, 2) == [-1, -1]
    assert R.choose([0.0, np.nan, 1.0], None, R.SIGMOID, 2) == [0, 1]
    assert R.choose([0.0, np.inf, 1.0], None, R.SIGMOID, 2) == [1, 2]
    assert R.choose([0.0, np.inf, 1.0], None, R.SOFTMAX, 2) == [0, 1]


def test_groups_by_hand():
    z = [0.0, 9.0, 5.0, 5.0, 1.0, 1.0]
    # best single 9 (group 0), best pair 5 + 5 (group 1)
    assert R.choose(z, None, R.SOFTMAX, 2, groups=3, kept=1) == [1, 0]
    assert R.choose(np.array(z) / 10, [0.0] * 6, R.SIGMOID, 2, 3, 1, 2) == [2, 3]
    # a group with one expert left is scored by that one
    assert R.choose([3.0, -np.inf, 1.0, 1.0], [0.0] * 4, R.SIGMOID, 1, 2, 1, 2) == [2]
    assert R.choose([9.0, -np.inf, -9.0, -9.0], [0.0] * 4, R.SIGMOID, 2, 2, 1, 2) == [0, -1]


def test_weights_sum_to_the_scale():
    z = np.array([-200.0, -210.0, 3.0, -205.0])
    for score in (R.SOFTMAX, R.SIGMOID):
        w, _ = R.weights(z, [0, 3, -1], score, True, 2.5)
        assert w[2] == 0 and w[:2].sum() == pytest.approx(2.5, rel=1e-14)
        assert w[0] / w[1] == pytest.approx(np.exp(5.0), rel=1e-12)
    w, _ = R.weights([0.0, np.log(3.0)], [1], R.SOFTMAX, False, 1.0)
    assert w[0] == pytest.approx(0.75, rel=1e-14)
    w, _ = R.weights([0.0, np.log(3.0)], [1], R.SIGMOID, False, 1.0)
    assert w[0] == pytest.approx(0.75, rel=1e-14)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(7)
    z, idx, dw = rng.standard_normal(6), [4, 1, -1], rng.standard_normal(3)
    dz, _ = R.gradient(z, idx, dw, score, renorm, 1.5)
    h = 1e-5
    for e in range(6):
        up, down = z.copy(), z.copy()
        up[e] += h
        down[e] -= h
        f = lambda v: (R.weights(v, idx, score, renorm, 1.5)[0] * dw).sum()
        # central differences: off by h^2 / 6 third derivatives (of order 1)
        assert abs((f(up) - f(down)) / (2 * h) - dz[e]) < 1e-8


def test_places_sort_the_slots():
    idx = np.array([[2, 0], [-1, 2], [0, 2]])
    off, pos = R.places(idx, 3)
    assert off.tolist() == [0, 2, 2, 5]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, 4]]


def test_exchange_by_hand():
    pos = np.array([[1, -1], [0, 2]])
    x = np.array([[1.0], [2.0]])
    assert R.gather(x, pos, np.full((4, 1), 9.0))[:, 0].tolist() == [2, 1, 2, 9]
    y, w = np.array([[1.0], [10.0], [100.0], [5.0]]), np.array([[2.0, 7.0], [3.0, -1.0]])
    r, m = R.combine(y, pos, w)
    assert r[:, 0].tolist() == [20.0, -97.0] and m[:, 0].tolist() == [20.0, 103.0]
    dy, dw, _ = R.combine_bwd(x, y, pos, w, np.full((4, 1), 9.0))
    assert dy[:, 0].tolist() == [6.0, 2.0, -2.0, 9.0]
    assert dw.tolist() == [[10.0, 0.0], [2.0, 200.0]]

"""Pins of the routing oracle: cases worked by hand, invariants, and its gradient
against differences."""
import math

import numpy as np
import pytest

from oracle import route

NINF = -math.inf


def test_softmax_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = route.route(x, 2, renorm=False)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = route.route(x, 3, renorm=True, scale=2.0)
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, [[8 / 7, 4 / 7, 2 / 7]])     # tie 0, 3: the lowest index


def test_sigmoid_bias_and_groups_by_hand():
    s = np.array([0.9, 0.1, 0.5, 0.6, 0.2, 0.3, 0.8, 0.05])
    x = np.log(s / (1 - s))[None]
    ids, w = route.route(x, 2, sigmoid=True, renorm=False)
    assert ids.tolist() == [[0, 6]] and np.allclose(w, [[0.9, 0.8]])
    bias = np.array([0, 0, 0, .35, 0, 0, 0, 0.0])
    ids, w = route.route(x, 2, bias=bias, sigmoid=True, renorm=True)
    assert ids.tolist() == [[3, 0]] and np.allclose(w, [[0.6 / 1.5, 0.9 / 1.5]])
    # groups of two: sums of both 1.0, 1.1, 0.5, 0.85; of the best 0.9, 0.6, 0.3, 0.8
    ids, _ = route.route(x, 3, sigmoid=True, groups=4, topk_groups=2, group_top=2)
    assert ids.tolist() == [[0, 3, 2]]
    ids, _ = route.route(x, 3, sigmoid=True, groups=4, topk_groups=2, group_top=1)
    assert ids.tolist() == [[0, 6, 1]]


def test_masked_nan_and_padding():
    x = np.array([[NINF, 1.0, NINF, 0.0], [NINF] * 4, [0.0, math.nan, 1.0, NINF], [0, 1, 2, 3.0]])
    ids, w = route.route(x, 3, live=3)
    assert ids.tolist() == [[1, 3, -1], [-1] * 3, [2, 0, 1], [-1] * 3]
    assert np.allclose(w[0], [math.e / (1 + math.e), 1 / (1 + math.e), 0]) and not w[1].any() and not w[3].any()
    assert np.isnan(w[2]).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(sigmoid, renorm):
    g = np.random.default_rng(7)
    T, E, k = 4, 9, 3
    x = g.standard_normal((T, E))
    x[1, 4] = NINF
    ids, _ = route.route(x, k, sigmoid=sigmoid)
    ids[2, 1] = -1
    ids[3, 2] = ids[3, 0]                     # an expert that is there twice
    dw = g.standard_normal((T, k))
    d, _ = route.route_backward(dw, x, ids, sigmoid, renorm, 1.5)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if x[t, e] == NINF:
                assert d[t, e] == 0
                continue
            up, dn = x[t].copy(), x[t].copy()
            up[e] += h
            dn[e] -= h
            num = (route.weights_of(up, ids[t], sigmoid, renorm, 1.5) -
                   route.weights_of(dn, ids[t], sigmoid, renorm, 1.5)) @ dw[t] / (2 * h)
            # central differences: h^2 of the third derivative (below 10 here), and 2^-52 / h of the values
            assert abs(num - d[t, e]) <= 1e-11 + 4 * 2.0 ** -52 / h * (np.abs(dw[t]).sum() * 1.5)

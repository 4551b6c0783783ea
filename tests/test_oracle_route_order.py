"""Without a bias experts go by their logits, also where their scores are equal numbers
in 64 bits; only the groups are told apart by scores.  Worked by hand."""
import math

import numpy as np
import pytest

from oracle import route

NINF = -math.inf


@pytest.mark.parametrize("group_top", [1, 2])
def test_saturated_sigmoids_go_by_logit(group_top):
    # sigmoids of 38 and more are 1 in 64 bits; the first group counts 1 or 2, the second 0.5 or 1
    x = np.array([[40.0, 41.0, 42.0, 1.0, 0.0, 0.0, 0.0, 0.0]])
    ids, w = route.route(x, 2, sigmoid=True, groups=2, topk_groups=1, group_top=group_top)
    assert ids.tolist() == [[2, 1]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("group_top", [1, 2])
def test_scores_of_zero_go_by_logit(group_top):
    # softmax: -900 and -800 below the largest are 0 in 64 bits
    x = np.array([[0.5, 0.0, -900.0, -800.0, -1.0, -1.0, -2.0, NINF]])
    ids, w = route.route(x, 4, groups=2, topk_groups=1, group_top=group_top)
    assert ids.tolist() == [[0, 1, 3, 2]] and w[0, 2:].tolist() == [0.0, 0.0]


def test_groups_of_equal_scores_go_by_index():
    # both groups' sigmoids add up to 2 in 64 bits: the first one stays, whatever its logits
    x = np.array([[40.0, 41.0, 0.0, 50.0, 60.0, 0.0]])
    ids, _ = route.route(x, 3, sigmoid=True, groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[1, 0, 2]]


def test_with_a_bias_by_the_sum():
    x = np.array([[40.0, 41.0, 42.0, 1.0, 0.0, 0.0, 0.0, 0.0]])
    bias = np.array([0.5, 0.25, 0.25, 0, 0, 0, 0, 0])
    ids, _ = route.route(x, 3, bias=bias, sigmoid=True, groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[0, 1, 2]]        # 1.5, and a tie of 1.25 by index

"""Choices (by a bias) so far below a row's largest logit that their softmax scores are 0
in 64 bits: renormalised weights are 0, the gradient is that of the softmax of the chosen
logits.  Both are written out here: p = 1 / (1 + e^-1), and p (1 - p)."""
import math

import pytest
import torch

import block_scaled_precision_04_amd as bs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 4099])
def test_weights_and_gradient(T):
    x = torch.tensor([[0.0, -800.0, -801.0, 0.5, -0.5, 0.0, 1.0, 0.0]] * T).cuda()
    bias = torch.tensor([0.0, 3.0, 2.0, 0, 0, 0, 0, 0]).cuda()
    ids, w = bs.moe_route(x, 2, bias=bias)
    assert (ids.cpu() == torch.tensor([1, 2])).all() and not w.any()
    dw = torch.tensor([[1.0, 0.0]] * T).cuda()
    d = bs.moe_route_backward(dw, x, ids).cpu().double()
    p = 1.0 / (1.0 + math.exp(-1.0))
    # fp64 within, one rounding to fp32
    assert (d[:, 1] - p * (1 - p)).abs().max() <= 1.5 * 2.0 ** -24 * p and (d[:, 2] + p * (1 - p)).abs().max() <= 1.5 * 2.0 ** -24 * p
    assert not d[:, [0, 3, 4, 5, 6, 7]].any()

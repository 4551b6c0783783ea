"""Routing of many tokens (the form that takes four tokens a wave) against the oracle.

Some tens of different rows, spread over 4099 tokens in a fixed order, so that every
wave holds a mix of them; every token is compared with its row's result.  Tolerances
as in test_gpu_moe_route.py: weights carry 8 half steps of fp32; below 2^-126, which
logits 80 and more apart reach, fp32 numbers are multiples of 2^-149, so that the one
rounding to fp32 may be off by 2^-150 (5.22684e-43 for 5.22793e-43: 1.1e-46 of 7.0e-46)."""
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from oracle import route
from tests.test_gpu_moe_route import H, _bias, _logits

pytestmark = pytest.mark.gpu
T = 4099


def _close(w, want):
    got = w.cpu().numpy().astype(np.float64)
    assert (np.isnan(got) == np.isnan(want)).all()
    bad = ~(np.abs(got - want) <= 8 * H * np.abs(want) + 2.0 ** -150) & ~np.isnan(want)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def _spread(x, seed=0):
    """[T, E] rows of x on the GPU, and the row of each."""
    at = np.random.default_rng(seed).integers(0, x.shape[0], T)
    return x[torch.from_numpy(at).to(x.device)].contiguous(), at


def _check(x, xo, k, b=None, bo=None, sigmoid=False, groups=1, keep=1, top=1, renorm=True, scale=1.0, seed=0):
    many, at = _spread(x, seed)
    ids, w = bs.moe_route(many, k, bias=b, score=int(sigmoid), groups=groups, topk_groups=keep, group_top=top,
                          renorm=renorm, scale=scale)
    io, wo = route.route(xo, k, bo, sigmoid, groups, keep, top, renorm, scale)
    bad = np.argwhere((ids.cpu().numpy() != io[at]).any(1))
    assert not len(bad), (len(bad), at[bad[0]], ids[int(bad[0, 0])].tolist(), io[at[bad[0, 0]]])
    _close(w, wo[at])


CASES = [   # E, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1), (3, 2, 1, 1, 1), (8, 8, 1, 1, 1), (16, 4, 4, 2, 2), (60, 4, 1, 1, 1), (64, 8, 16, 4, 2),
    (64, 6, 8, 3, 1), (65, 6, 1, 1, 1), (96, 5, 3, 2, 2), (128, 8, 1, 1, 1), (128, 1, 8, 1, 2), (128, 8, 16, 5, 2),
    (160, 6, 8, 3, 1), (250, 7, 1, 1, 1), (256, 8, 1, 1, 1), (256, 8, 8, 4, 2), (256, 8, 2, 1, 2), (256, 3, 16, 9, 2),
    (256, 8, 4, 4, 1), (257, 8, 1, 1, 1), (240, 8, 15, 4, 2), (256, 9, 8, 4, 2),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route(case, sigmoid, dtype):
    E, k, G, keep, top = case
    for kind, with_bias, renorm in (("normal", True, True), ("few", False, False), ("masked", True, False),
                                    ("few", True, True), ("masked", False, True), ("normal", False, True),
                                    ("wide", False, True)):
        x, xo = _logits(E, 50, E, dtype, kind)
        b, bo = _bias(E, E) if with_bias else (None, None)
        _check(x, xo, k, b, bo, sigmoid, G, keep, top, renorm, 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups", [(64, 4), (128, 1), (256, 8)])
def test_values_that_fp32_cannot_tell_apart(sigmoid, E, groups):
    """Runs of two to all of a token's values within an fp32 step of each other, with
    biases and without."""
    g = np.random.default_rng(E)
    x = (g.standard_normal((60, E)) * 1.5).astype(np.float32)
    for t in range(60):
        n = (2, 3, 4, 5, 8, 13, E)[t % 7]
        at = g.permutation(E)[:n]
        x[t, at] = 2.0 + g.integers(-8, 9, n) * 2.0 ** -22
    dx = torch.from_numpy(x).cuda()
    b = (g.integers(-3, 4, E) * 2.0 ** -25).astype(np.float32)
    for bias in (None, b, b + np.float32(1.0)):
        for k in (2, 8):
            _check(dx, x.astype(np.float64), k, None if bias is None else torch.from_numpy(bias).cuda(),
                   None if bias is None else bias.astype(np.float64), sigmoid, groups, max(1, groups // 2),
                   2 if groups > 1 else 1)


@pytest.mark.parametrize("lanes", ["one lane", "spread"])
def test_many_picks_of_neighbours(lanes):
    """The largest values side by side (16 experts of one lane), and just unequal."""
    g = np.random.default_rng(1)
    x = (g.standard_normal((40, 256)) - 3.0).astype(np.float32)
    for t in range(40):
        at = 16 * (t % 16) + np.arange(16) if lanes == "one lane" else np.arange(16) * 16 + t % 16
        x[t, at] = 1.0 + g.permutation(16) * np.float32(2.0 ** -23 if t % 2 else 2.0 ** -21)
    dx = torch.from_numpy(x).cuda()
    b = np.zeros(256, np.float32)
    for sigmoid in (False, True):
        _check(dx, x.astype(np.float64), 8, None, None, sigmoid)
        _check(dx, x.astype(np.float64), 8, torch.from_numpy(b).cuda(), b.astype(np.float64), sigmoid)


@pytest.mark.parametrize("big", [1000.0, 1e6])
@pytest.mark.parametrize("k,keep", [(8, 4), (1, 1), (2, 2)])
def test_group_sums_of_large_biases_that_cancel(big, k, keep):
    x = torch.randn((200, 256), generator=torch.Generator().manual_seed(5)).cuda()
    b = np.full(256, -big)
    b[np.arange(8) * 32 + np.arange(8)] = big
    bias = torch.from_numpy(b.astype(np.float32)).cuda()
    _check(x, x.double().cpu().numpy(), k, bias, b, True, 8, keep, 2)


def test_nan_and_inf():
    x = torch.randn((12, 64), generator=torch.Generator().manual_seed(1))
    x[0, 3] = math.nan
    x[1, 5] = math.inf
    x[2, :] = math.nan
    x[3, :30] = -math.inf
    x[4, 1], x[4, 2], x[4, 9] = math.nan, math.inf, -math.inf
    x[5, :] = -math.inf
    x[6, :60] = -math.inf
    for sigmoid in (False, True):
        for bias in (None, torch.linspace(-.2, .2, 64), torch.linspace(-.2, .2, 64).masked_fill(torch.arange(64) % 5 == 0, -math.inf),
                     torch.linspace(-.2, .2, 64).masked_fill(torch.arange(64) == 7, math.inf)):
            for groups in (1, 4):
                _check(x.cuda(), x.double().numpy(), 6, None if bias is None else bias.cuda(),
                       None if bias is None else bias.double().numpy(), sigmoid, groups, min(groups, 2), 1)


@pytest.mark.parametrize("live", [0, 1, 4, 4093, 4098, 4099, 5000, -1])
def test_padding_tokens(live):
    x, xo = _logits(7, 30, 64, "fp32")
    many, at = _spread(x)
    if live < T:
        many[max(live, 0):] = math.nan
    ids, w = bs.moe_route(many, 6, rows=torch.tensor([live], dtype=torch.int32, device="cuda"))
    io, wo = route.route(xo, 6)
    n = min(max(live, 0), T)
    got = ids.cpu().numpy()
    assert np.array_equal(got[:n], io[at[:n]]) and (got[n:] == -1).all() and not w[n:].any()
    _close(w[:n], wo[at[:n]])


def test_strided_logits_and_odd_addresses():
    base = torch.randn((T, 300), generator=torch.Generator().manual_seed(3)).cuda()
    bias = (torch.randn(260, generator=torch.Generator().manual_seed(4)) * 0.1).cuda()
    for dt in (torch.float32, torch.bfloat16):
        b = base.to(dt)
        for lo, hi in ((0, 256), (1, 257), (4, 132), (8, 72), (3, 254)):
            view = b[:, lo:hi]
            for o in (0, 1, 4):
                ids, w = bs.moe_route(view, 7, bias=bias[o:o + hi - lo], score=bs.BS_SCORE_SIGMOID)
                whole = bs.moe_route(view[:64].contiguous(), 7, bias=bias[o:o + hi - lo].clone(), score=bs.BS_SCORE_SIGMOID)
                assert torch.equal(ids[:64], whole[0])
                at = np.arange(0, T, 37)
                io, wo = route.route(view.double().cpu().numpy()[at], 7, bias[o:o + hi - lo].double().cpu().numpy(), True)
                assert np.array_equal(ids.cpu().numpy()[at], io)
                _close(w[torch.from_numpy(at).cuda()], wo)


def test_a_token_s_result_does_not_depend_on_how_many_there_are():
    x = torch.randn((T, 256), generator=torch.Generator().manual_seed(9)).cuda()
    bias = (torch.randn(256, generator=torch.Generator().manual_seed(8)) * 0.1).cuda()
    for kw in (dict(), dict(bias=bias, score=bs.BS_SCORE_SIGMOID, groups=8, topk_groups=4, group_top=2, scale=2.5),
               dict(renorm=False)):
        ids, w = bs.moe_route(x, 8, **kw)
        parts = [bs.moe_route(x[i:i + 1000], 8, **kw) for i in range(0, T, 1000)]
        assert torch.equal(ids, torch.cat([i for i, _ in parts]))
        assert torch.allclose(w, torch.cat([v for _, v in parts]), rtol=16 * 2.0 ** -24, atol=0)

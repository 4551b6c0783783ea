"""Routing to experts and its gradient against the oracle.

ids are whole numbers and equal.  weights: an exponential (2 ulps), the sum over
the scores (2 half steps), a quotient, a product with scale, one rounding each: 8
half steps of fp32.  dlogits: every term of the oracle's sum of magnitudes carries
the weights' error and up to 8 roundings more: 16 half steps; and one rounding to
the output's type."""
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from oracle import route

pytestmark = pytest.mark.gpu
H = 2.0 ** -24
HOUT = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _logits(seed, T, E, dtype, kind="normal"):
    g = np.random.default_rng(seed)
    if kind == "few":                        # many equal logits
        x = g.integers(-3, 4, (T, E)) * 0.5
    elif kind == "wide":
        x = g.standard_normal((T, E)) * 30
    else:
        x = g.standard_normal((T, E)) * 1.5 + g.standard_normal(E)
    if kind == "masked":
        x = np.where(g.random((T, E)) < 0.6, -math.inf, x)
        x[0] = -math.inf
    t = torch.tensor(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.cuda(), t.double().numpy()


def _bias(seed, E):
    b = (np.random.default_rng(seed).standard_normal(E) * 0.1).astype(np.float32)
    return torch.from_numpy(b).cuda(), b.astype(np.float64)


def _close(w, want):
    got = w.cpu().numpy().astype(np.float64)
    assert (np.isnan(got) == np.isnan(want)).all()
    bad = ~(np.abs(got - want) <= 8 * H * np.abs(want)) & ~np.isnan(want)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


CASES = [
    # T, E, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (3, 8, 2, 1, 1, 1), (5, 64, 64, 1, 1, 1), (17, 60, 4, 1, 1, 1), (9, 65, 6, 1, 1, 1),
    (33, 256, 8, 1, 1, 1), (64, 256, 8, 8, 4, 2), (20, 160, 6, 8, 3, 1), (7, 96, 5, 3, 2, 2), (6, 128, 8, 64, 9, 1),
    (6, 128, 8, 64, 9, 2), (12, 512, 10, 16, 16, 2), (4, 1024, 64, 2, 1, 2), (5, 1000, 8, 40, 7, 2), (2, 257, 9, 1, 1, 1),
    (130, 16, 16, 4, 4, 2), (10, 12, 3, 12, 5, 1), (8, 384, 8, 1, 1, 1), (3, 513, 64, 27, 10, 2), (2, 30, 7, 5, 3, 2),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route(case, sigmoid, dtype):
    T, E, k, G, keep, top = case
    for kind, with_bias, renorm in (("normal", True, True), ("few", False, False), ("masked", True, False),
                                    ("few", True, True), ("masked", False, True), ("normal", False, True)):
        x, xo = _logits(T + E, T, E, dtype, kind)
        b, bo = _bias(E, E) if with_bias else (None, None)
        score = bs.BS_SCORE_SIGMOID if sigmoid else bs.BS_SCORE_SOFTMAX
        ids, w = bs.moe_route(x, k, bias=b, score=score, groups=G, topk_groups=keep, group_top=top, renorm=renorm,
                              scale=2.5)
        io, wo = route.route(xo, k, bo, sigmoid, G, keep, top, renorm, 2.5)
        assert np.array_equal(ids.cpu().numpy(), io), (kind, with_bias, renorm)
        _close(w, wo)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_scores_that_fp32_cannot_tell_apart(sigmoid):
    """Scores and biases whose sums differ by less than an fp32 step, in every order."""
    g = np.random.default_rng(4)
    T, E = 64, 128
    x = (0.5 + g.integers(-8, 9, (T, E)) * 2.0 ** -24).astype(np.float32)
    s0 = 1 / (1 + math.exp(-.5)) if sigmoid else 1 / E
    b = (1.0 - s0 + g.integers(-3, 4, E) * 2.0 ** -25).astype(np.float32)
    ids, w = bs.moe_route(torch.from_numpy(x).cuda(), 16, bias=torch.from_numpy(b).cuda(),
                          score=bs.BS_SCORE_SIGMOID if sigmoid else bs.BS_SCORE_SOFTMAX, groups=4, topk_groups=2,
                          group_top=2)
    io, wo = route.route(x, 16, b, sigmoid, 4, 2, 2)
    assert np.array_equal(ids.cpu().numpy(), io)
    _close(w, wo)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_wide_logits(sigmoid, dtype):
    """Scores that fp32 holds as equal (sigmoids next to one) or as zero."""
    x, xo = _logits(3, 40, 96, dtype, "wide")
    for b, bo in ((None, None), _bias(1, 96)):
        ids, w = bs.moe_route(x, 8, bias=b, score=int(sigmoid), renorm=not sigmoid)
        io, wo = route.route(xo, 8, bo, sigmoid, renorm=not sigmoid)
        assert np.array_equal(ids.cpu().numpy(), io)
        got = w.cpu().numpy()
        assert (np.abs(got - wo) <= 8 * H * np.abs(wo) + 2.0 ** -126).all()


def test_nan_and_inf():
    x = torch.randn((6, 32), generator=torch.Generator().manual_seed(1))
    x[0, 3] = math.nan
    x[1, 5] = math.inf
    x[2, :] = math.nan
    x[3, :30] = -math.inf
    x[4, 1], x[4, 2], x[4, 9] = math.nan, math.inf, -math.inf
    for sigmoid in (False, True):
        for bias in (None, torch.linspace(-.2, .2, 32)):
            for groups in (1, 4):
                ids, w = bs.moe_route(x.cuda(), 4, bias=None if bias is None else bias.cuda(), score=int(sigmoid),
                                      groups=groups, topk_groups=min(groups, 2), group_top=1)
                io, wo = route.route(x.double().numpy(), 4, None if bias is None else bias.double().numpy(), sigmoid,
                                     groups, min(groups, 2), 1)
                assert np.array_equal(ids.cpu().numpy(), io), (sigmoid, bias is None, groups)
                _close(w, wo)


def test_bias_that_switches_off():
    x, xo = _logits(2, 10, 48, "fp32")
    b = torch.zeros(48)
    b[::3] = -math.inf
    b[1] = math.inf
    ids, w = bs.moe_route(x, 40, bias=b.cuda(), score=bs.BS_SCORE_SIGMOID)
    io, wo = route.route(xo, 40, b.double().numpy(), True)
    assert np.array_equal(ids.cpu().numpy(), io) and (io == -1).any()
    _close(w, wo)


@pytest.mark.parametrize("k,keep", [(8, 4), (1, 1), (2, 2)])
@pytest.mark.parametrize("big", [100.0, 1000.0, 1e6])
def test_group_sums_of_large_biases_that_cancel(big, k, keep):
    """Of each group one expert has +big and the others -big: fp32 sums of the two
    largest lose the scores that decide between the groups."""
    T, E, groups = 200, 256, 8
    x = torch.randn((T, E), generator=torch.Generator().manual_seed(5)).cuda()
    b = np.full(E, -big)
    b[np.arange(groups) * 32 + np.arange(groups)] = big
    bias = torch.from_numpy(b.astype(np.float32)).cuda()
    ids, w = bs.moe_route(x, k, bias=bias, score=bs.BS_SCORE_SIGMOID, groups=groups, topk_groups=keep, group_top=2)
    want, ww = route.route(x.double().cpu().numpy(), k, bias.double().cpu().numpy(), True, groups, keep, 2)
    assert np.array_equal(ids.cpu().numpy(), want)
    _close(w, ww)


@pytest.mark.parametrize("k", [2, 3, 8, 12])
@pytest.mark.parametrize("bias", [0.0, 1000.0])
def test_the_last_two_picks_closer_than_fp32(k, bias):
    """The k-th value just below the (k-1)-th and, by its index, before it where fp32
    holds them equal; all others far away."""
    T, E = 64, 64
    g = np.random.default_rng(k)
    x = np.full((T, E), -4.0, np.float32)
    for t in range(T):
        at = np.sort(g.permutation(E)[:k])
        x[t, at] = 1.0 + 0.25 * np.arange(k)
        lo, hi = at[0], at[1]
        v = np.float32(-1.0 + 0.01 * t)
        x[t, lo], x[t, hi] = v, v + np.float32(2.0 ** -21 if bias == 0.0 else 1e-5)
    b = np.full(E, bias, np.float32)
    dx = torch.from_numpy(x).cuda()
    ids, w = bs.moe_route(dx, k, bias=torch.from_numpy(b).cuda(), score=bs.BS_SCORE_SIGMOID)
    want, ww = route.route(x.astype(np.float64), k, b.astype(np.float64), True)
    assert np.array_equal(ids.cpu().numpy(), want)
    _close(w, ww)


@pytest.mark.parametrize("live", [0, 1, 5, 9, 20, -1])
def test_padding_tokens(live):
    x, xo = _logits(5, 9, 64, "bf16")
    x[max(live, 0):] = math.nan
    ids, w = bs.moe_route(x, 6, rows=torch.tensor([live], dtype=torch.int32, device="cuda"))
    n = min(max(live, 0), 9)
    io, wo = route.route(xo, 6, live=n)
    assert np.array_equal(ids.cpu().numpy(), io)
    _close(w, wo)


def test_padded_rows_of_logits_and_outputs():
    base = torch.randn((20, 100), generator=torch.Generator().manual_seed(3)).cuda()
    for dt in (torch.float32, torch.bfloat16):
        b = base.to(dt)
        for view in (b[:, 1:65], b[::2, 3:90], b[4:5, 7:71]):
            T, E = view.shape
            ids = torch.empty((T, 5), dtype=torch.int32, device="cuda")
            w = torch.empty((T, 5), device="cuda")
            out = bs.moe_route(view, 5, ids=ids, weights=w)
            assert out[0] is ids and out[1] is w
            io, wo = route.route(view.double().cpu().numpy(), 5)
            assert np.array_equal(ids.cpu().numpy(), io)
            _close(w, wo)
            d = torch.full((T, E + 3), 7.0, dtype=dt, device="cuda")
            bs.moe_route_backward(torch.ones((T, 5), device="cuda"), view, ids, renorm=False, dlogits=d[:, :E])
            assert bool((d[:, E:] == 7.0).all())
            _grad_close(d[:, :E], torch.ones((T, 5)), view, ids, False, False, 1.0)


# ------------------------------------------------------------------ the gradient
def _grad_close(d, dw, x, ids, sigmoid, renorm, scale):
    want, mag = route.route_backward(dw.cpu().double().numpy(), x.double().cpu().numpy(), ids.cpu().numpy(), sigmoid,
                                     renorm, scale)
    got = d.double().cpu().numpy()
    h = 2.0 ** -8 if d.dtype == torch.bfloat16 else 2.0 ** -24
    bad = ~(np.abs(got - want) <= 16 * H * mag + h * np.abs(want) * (1 + 16 * H) + 2.0 ** -133)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (5, 64, 64), (17, 60, 4), (9, 65, 6), (33, 256, 8), (7, 100, 10),
                                   (4, 1000, 8), (2, 1024, 64), (3, 513, 9), (70, 16, 3), (6, 384, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_backward(T, E, k, sigmoid, renorm, dtype):
    g = torch.Generator().manual_seed(T + E)
    for kind in ("normal", "masked", "few"):
        x, _ = _logits(E, T, E, dtype, kind)
        ids, _ = bs.moe_route(x, k, score=int(sigmoid))
        dw = torch.randn((T, k), generator=g)
        d = bs.moe_route_backward(dw.cuda(), x, ids, score=int(sigmoid), renorm=renorm, scale=2.5)
        assert d.dtype == x.dtype
        _grad_close(d, dw, x, ids, sigmoid, renorm, 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_repeated_and_absent_ids(sigmoid, renorm):
    g = torch.Generator().manual_seed(1)
    T, E, k = 12, 40, 7
    x = torch.randn((T, E), generator=g).cuda()
    ids = torch.randint(-2, E + 2, (T, k), generator=g, dtype=torch.int32)
    ids[0] = -1
    ids[1] = 5
    ids[2, :4] = 9
    ids[3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1, 1, 2, 2, 3])
    ids = ids.cuda()
    dw = torch.randn((T, k), generator=g)
    dw[ids.cpu() == -1] = math.nan               # the gradient of a weight that is not there is not used
    d = bs.moe_route_backward(dw.cuda(), x, ids, score=int(sigmoid), renorm=renorm)
    _grad_close(d, torch.nan_to_num(dw), x, ids, sigmoid, renorm, 1.0)
    again = bs.moe_route_backward(dw.cuda(), x, ids, score=int(sigmoid), renorm=renorm)
    assert torch.equal(d, again)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_is_the_slope_of_the_forward(sigmoid, renorm):
    """Differences of moe_route itself, the choice unchanged by the step."""
    g = torch.Generator().manual_seed(2)
    E, k, step = 16, 16, 2.0 ** -7
    x = torch.randn((1, E), generator=g).cuda()
    ids, _ = bs.moe_route(x, k, score=int(sigmoid))
    dw = torch.randn((1, k), generator=g).cuda()
    d = bs.moe_route_backward(dw, x, ids, score=int(sigmoid), renorm=renorm)[0].double()
    by_expert = torch.zeros(E, device="cuda").scatter_(0, ids[0].long(), dw[0]).double()
    for e in range(E):
        val = []
        for sgn in (1, -1):
            y = x.clone()
            y[0, e] += sgn * step
            i, w = bs.moe_route(y, k, score=int(sigmoid), renorm=renorm)
            val.append((by_expert[i[0].long()] * w[0].double()).sum())
        num = (val[0] - val[1]) / (2 * step)
        # step^2 / 6 of a third derivative below 8 |dw|, and 8 half steps of each weight
        tol = step * step / 6 * 8 * dw.abs().sum() + 8 * H * dw.abs().sum() / step + H * abs(float(x[0, e])) / step * abs(d[e])
        assert abs(num - d[e]) <= tol, (e, float(num), float(d[e]))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_of_padding_tokens_is_zero(sigmoid, renorm, dtype):
    """Whatever their logits hold (NaN, infinities) and dweights, rows without a choice get zeros."""
    x, _ = _logits(3, 9, 40, dtype)
    x[4:] = math.nan
    x[5] = math.inf
    x[6] = -math.inf
    ids, w = bs.moe_route(x, 4, score=int(sigmoid), renorm=renorm, rows=torch.tensor([4], dtype=torch.int32, device="cuda"))
    dw = torch.randn((9, 4), generator=torch.Generator().manual_seed(1)).cuda()
    dw[7] = math.nan
    d = bs.moe_route_backward(dw, x, ids, score=int(sigmoid), renorm=renorm, dlogits=torch.full_like(x, 7.0))
    assert not d[4:].any() and d[:4].isfinite().all()
    _grad_close(d[:4], dw[:4], x[:4], ids[:4], sigmoid, renorm, 1.0)


def test_empty():
    x = torch.empty((0, 32), device="cuda")
    ids, w = bs.moe_route(x, 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert bs.moe_route_backward(w, x, ids).shape == (0, 32)

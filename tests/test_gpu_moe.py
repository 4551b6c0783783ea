"""Expert sort, row gather, weighted combine and its gradient against the oracle.

Tolerances: sorts are equal; gathered rows are bit-equal; combine rounds an
fp32 sum of k terms (k - 1 additions and k products, 2^-24 each of the sum of
magnitudes) once to bf16 (2^-8); dy is one fp32 product (exact to 2^-24) and one
bf16 rounding; dweights is an fp32 sum of K terms, at most K additions each
2^-24 of the sum of magnitudes (products are exact to 2^-24)."""
import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from block_scaled_precision_04_amd import synth
from oracle import codecs, mxfp4
from tests.gpu_util import dev_bf16, host_bits16

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda() if dtype is None else torch.tensor(a, dtype=dtype).cuda()


def _ids(seed, T, k, E, drop=0.0, skew=False):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, (T, k))
    if skew:
        ids = np.minimum(ids, g.integers(0, max(1, E // 8) + 1, (T, k)))
    if drop:
        out = g.random((T, k)) < drop
        ids = np.where(out, g.choice([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1], (T, k)), ids)
    return ids.astype(np.int32)


def _sort(ids, E):
    T, k = ids.shape
    r, p, o = bs.moe_sort(_dev(ids), E, ws=bs.alloc_workspace(bs.BS_OP_MOE_SORT, T, k, E))
    torch.cuda.synchronize()
    return r, p, o


SORTS = [(1, 1, 1, 0, False), (1, 8, 256, 0, False), (8, 8, 256, 0, False), (3, 5, 7, .5, False), (64, 1, 2, 0, True),
         (65, 1, 1024, .2, False), (1000, 8, 256, .1, True), (1024, 8, 1000, 0, False), (1025, 8, 33, .3, False),
         (8191, 3, 256, 0, True), (40000, 8, 256, .25, False), (130001, 9, 64, 0, False), (7, 4, 16, 1.0, False),
         (9000, 2, 5, 1.0, False),
         (4096, 1, 200, 0, False), (4097, 1, 200, .1, False), (2049, 2, 3, 0, True), (270000, 1, 40, .1, True)]


@pytest.mark.parametrize("T,k,E,drop,skew", SORTS)
def test_sort(T, k, E, drop, skew):
    ids = _ids(T + k + E, T, k, E, drop, skew)
    r, p, o = _sort(ids, E)
    flat = ids.reshape(-1).astype(np.int64)
    keep = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(keep, flat, E), kind="stable")
    n = int(keep.sum())
    rows = np.full(T * k, -1)
    rows[:n] = order[:n] // k
    pos = np.full(T * k, -1)
    pos[order[:n]] = np.arange(n)
    if T <= 1000:                                   # the oracle's list form, where it is quick
        ro, po, oo = mxfp4.moe_sort(ids, E)
        assert np.array_equal(ro, rows) and np.array_equal(po.reshape(-1), pos)
        assert np.array_equal(o.cpu().numpy(), oo)
    assert np.array_equal(o.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=E))]))
    assert np.array_equal(r.cpu().numpy(), rows)
    assert np.array_equal(p.cpu().numpy().reshape(-1), pos)


def test_sort_no_tokens():
    r, p, o = bs.moe_sort(torch.empty((0, 8), dtype=torch.int32, device="cuda"), 5)
    torch.cuda.synchronize()
    assert r.numel() == 0 and p.shape == (0, 8) and o.tolist() == [0] * 6


def test_sort_same_expert_for_all():
    ids = np.full((4100, 4), 3, np.int32)
    r, p, o = _sort(ids, 8)
    assert o.tolist() == [0, 0, 0, 0] + [16400] * 5
    assert np.array_equal(r.cpu().numpy(), np.arange(16400) // 4)


def test_sort_leaves_the_workspace_counters():
    """The workspace's counter region, which other calls rely on, stays zero."""
    ws = bs.alloc_workspace(bs.BS_OP_MOE_SORT, 5000, 8, 256)
    bs.moe_sort(_dev(_ids(1, 5000, 8, 256)), 256, ws=ws)
    torch.cuda.synchronize()
    assert not ws[: 64 * 1024].any()


ROWS = [(1, 1, 1, 8, 0), (1, 8, 256, 2048, 0), (8, 8, 256, 2048, 0), (5, 3, 4, 24, .4), (33, 10, 12, 1096, .2),
        (700, 8, 64, 2048, .25), (2100, 2, 8, 136, 0), (3, 9, 9, 32768, .3), (40, 17, 6, 264, .1), (6, 4, 8, 512, 1.0)]


def _rows_case(T, k, E, K, drop):
    ids = _ids(T * k + E, T, k, E, drop)
    _, pos, off = mxfp4.moe_sort(ids, E)
    g = synth.rng(T + K)
    w = g.standard_normal((T, k)).astype(np.float32)
    return pos, int(off[-1]), synth.bf16_normal(g, (T * k, K), 1.0), synth.bf16_normal(g, (T, K), 1.0), w


@pytest.mark.parametrize("T,k,E,K,drop", ROWS)
def test_gather(T, k, E, K, drop):
    pos, n, _, x, _ = _rows_case(T, k, E, K, drop)
    out = torch.full((T * k, K), 7.0, dtype=torch.bfloat16, device="cuda")
    bs.moe_gather(dev_bf16(x), _dev(pos), out=out)
    torch.cuda.synchronize()
    want = np.full((T * k, K), 0x40E0, np.uint16)          # 7.0: untouched
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[pos[t, j]] = x[t]
    assert np.array_equal(host_bits16(out), want)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,K,drop", ROWS)
def test_combine(T, k, E, K, drop, weighted):
    pos, n, y, _, w = _rows_case(T, k, E, K, drop)
    y[n:] = 0x7FC0                                          # rows of no pair: NaN, must not be read into sums
    out = bs.moe_combine(dev_bf16(y), _dev(pos), _dev(w) if weighted else None)
    torch.cuda.synchronize()
    want, mag = mxfp4.moe_combine(codecs.decode_bf16(y), pos, w if weighted else None)
    got = codecs.decode_bf16(host_bits16(out))
    d = 2 * k * 2.0 ** -24 * mag
    assert (np.abs(got - want) <= d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -134).all()
    none = (pos < 0).all(axis=1)
    assert (got[none] == 0).all()


@pytest.mark.parametrize("T,k,E,K,drop", ROWS)
def test_combine_backward(T, k, E, K, drop):
    pos, n, y, dout, w = _rows_case(T, k, E, K, drop)
    y[n:] = 0x7FC0
    dy = torch.full((T * k, K), 7.0, dtype=torch.bfloat16, device="cuda")
    bs_dy, dw = bs.moe_combine_backward(dev_bf16(dout), dev_bf16(y), _dev(pos), _dev(w), dy=dy)
    torch.cuda.synchronize()
    wy, ww, mag = mxfp4.moe_combine_backward(codecs.decode_bf16(dout), codecs.decode_bf16(y), pos, w)
    got = codecs.decode_bf16(host_bits16(bs_dy))
    free = np.isnan(wy).all(axis=1)
    free[n:] = True
    assert (got[free] == 7.0).all()
    e = np.abs(wy[~free])
    assert (np.abs(got[~free] - wy[~free]) <= (2.0 ** -8 + 2.0 ** -23) * e + 2.0 ** -134).all()
    assert (np.abs(dw.cpu().numpy() - ww) <= (K + 1) * 2.0 ** -24 * mag).all()
    assert (dw.cpu().numpy()[pos < 0] == 0).all()


def test_combine_ignores_positions_out_of_range():
    y = torch.ones((4, 8), dtype=torch.bfloat16, device="cuda")
    pos = _dev(np.array([[0, 4], [2 ** 31 - 1, -5]], np.int32))
    assert bs.moe_combine(y, pos).float().cpu().tolist() == [[1.0] * 8, [0.0] * 8]
    xs = torch.full((4, 8), 5.0, dtype=torch.bfloat16, device="cuda")
    bs.moe_gather(torch.ones((2, 8), dtype=torch.bfloat16, device="cuda"), pos, out=xs)
    assert xs.float().cpu()[:, 0].tolist() == [1.0, 5.0, 5.0, 5.0]


def test_gather_gradient_is_combine():
    """<moe_gather(x), d> = <x, moe_combine(d)> over the kept slots: exact
    integers, so the two sides are equal, and against a difference quotient."""
    g = np.random.default_rng(4)
    T, k, E, K = 19, 3, 5, 40
    ids = _ids(3, T, k, E, .2)
    r, pos, off = _sort(ids, E)
    n = int(off[-1])
    x = torch.tensor(g.integers(-4, 5, (T, K)), dtype=torch.bfloat16).cuda()
    d = torch.tensor(g.integers(-4, 5, (T * k, K)), dtype=torch.bfloat16).cuda()
    xs = torch.zeros((T * k, K), dtype=torch.bfloat16, device="cuda")
    bs.moe_gather(x, pos, out=xs)
    dx = bs.moe_combine(d, pos)
    lhs = (xs.double() * d.double())[:n].sum().item()
    assert lhs == (x.double() * dx.double()).sum().item()
    x2 = x.clone()
    x2[4, 7] += 2
    xs2 = xs.clone()
    bs.moe_gather(x2, pos, out=xs2)
    assert ((xs2.double() - xs.double()) * d.double())[:n].sum().item() / 2 == dx[4, 7].item()


def test_combine_gradient_against_differences():
    """Integer data keeps every sum exact, so the forward's differences are exact
    directional derivatives."""
    g = np.random.default_rng(5)
    T, k, E, K = 6, 4, 3, 16
    _, pos, off = _sort(_ids(5, T, k, E, .2), E)
    y = torch.tensor(g.integers(-3, 4, (T * k, K)), dtype=torch.bfloat16).cuda()
    w = torch.tensor(g.integers(-2, 3, (T, k)), dtype=torch.float32).cuda()
    dout = torch.tensor(g.integers(-2, 3, (T, K)), dtype=torch.bfloat16).cuda()
    dy, dw = bs.moe_combine_backward(dout, y, pos, w, dy=torch.zeros_like(y))
    f = lambda y_, w_: (bs.moe_combine(y_, pos, w_).double() * dout.double()).sum().item()
    for t in range(T):
        for j in range(k):
            e = torch.zeros_like(w)
            e[t, j] = 1
            assert f(y, w + e) - f(y, w) == dw[t, j].item()
    for s in range(0, T * k, 3):
        e = torch.zeros_like(y)
        e[s, 5] = 1
        assert f(y + e, w) - f(y, w) == dy[s, 5].item()

"""Pins of oracle/mxfp4.py to exact rationals, the printed e2m1 table and
differences of the forward definition."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mxfp4, codecs

TABLE = [Fraction(v) for v in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]


def _brute_code(v):
    """Nearest table entry of |v| <= anything, ties to the even index, saturating."""
    a = min(abs(v), Fraction(6))
    best = min(range(8), key=lambda i: (abs(TABLE[i] - a), i % 2))
    return best


def test_encode_against_brute_force():
    vals = [Fraction(i, 64) for i in range(0, 64 * 9)]
    got = mxfp4.encode_e2m1([float(v) for v in vals])
    assert got.tolist() == [_brute_code(v) for v in vals]
    neg = mxfp4.encode_e2m1([-float(v) for v in vals])
    assert (neg == (got | 8)).all()          # the sign of a zero is kept too


def test_quant_against_rationals():
    g = np.random.default_rng(1)
    x = g.standard_normal((40, 64)) * np.exp2(g.integers(-130, 126, (40, 1)).astype(float))
    x = codecs.decode_bf16(codecs.round_to_bf16(x))
    x[0, :32] = 0.0
    x[1, 3] = 2.0 ** -133                    # the smallest bf16
    q, s = mxfp4.quant_mxfp4(x)
    codes = codecs.unpack_fp4(q)
    for m in range(x.shape[0]):
        for b in range(2):
            blk = [Fraction(float(v)) for v in x[m, 32 * b:32 * b + 32]]
            amax = max(abs(v) for v in blk)
            e = -127
            if amax:
                e = -200
                while Fraction(2) ** (e + 1) <= amax:
                    e += 1
                e = max(e - 2, -127)
            assert s[m, b] == e + 127
            for i, v in enumerate(blk):
                assert int(codes[m, 32 * b + i]) & 7 == _brute_code(v / Fraction(2) ** e)


def test_quant_not_finite():
    x = np.ones((1, 96))
    x[0, 5] = np.inf
    x[0, 40] = np.nan
    q, s = mxfp4.quant_mxfp4(x)
    assert s.tolist() == [[255, 255, 125]] and not q[0, :32].any() and q[0, 32:].all()


def test_sort_small_by_hand():
    rows, pos, offsets = mxfp4.moe_sort(np.array([[2, 0], [0, -1], [7, 2]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert rows.tolist() == [0, 1, 0, 2, -1, -1]
    assert pos.tolist() == [[2, 0], [1, -1], [-1, 3]]


def test_combine_gradient_against_differences():
    g = np.random.default_rng(2)
    ids = np.array([[0, 1, 1], [2, -1, 0], [-1, -1, -1]])
    _, pos, _ = mxfp4.moe_sort(ids, 3)
    y, w, dout = g.standard_normal((9, 4)), g.standard_normal((3, 3)), g.standard_normal((3, 4))
    f = lambda y_, w_: float((mxfp4.moe_combine(y_, pos, w_)[0] * dout).sum())
    dy, dw, _ = mxfp4.moe_combine_backward(dout, y, pos, w)
    h = 1e-6
    for idx in np.ndindex(y.shape):
        d = np.zeros_like(y)
        d[idx] = h
        num = (f(y + d, w) - f(y - d, w)) / (2 * h)
        assert num == pytest.approx(0.0 if np.isnan(dy[idx]) else dy[idx], abs=1e-8)
    for idx in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[idx] = h
        assert (f(y, w + d) - f(y, w - d)) / (2 * h) == pytest.approx(dw[idx], abs=1e-8)


def test_w4a4_against_rationals():
    g = np.random.default_rng(3)
    M, N, K = 2, 3, 64
    ap, wp = g.integers(0, 256, (M, K // 2), dtype=np.uint8), g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    ae, we = g.integers(110, 140, (M, 2), dtype=np.uint8), g.integers(110, 140, (N, 2), dtype=np.uint8)
    c, _ = mxfp4.w4a4_gemm(ap, ae, wp, we)
    sgn = lambda code: -TABLE[code & 7] if code & 8 else TABLE[code & 7]
    val = lambda p, e, r, k: sgn((int(p[r, k // 2]) >> (4 * (k % 2))) & 15) * Fraction(2) ** (int(e[r, k // 32]) - 127)
    for m in range(M):
        for n in range(N):
            want = sum(val(ap, ae, m, k) * val(wp, we, n, k) for k in range(K))
            assert c[m, n] == pytest.approx(float(want), rel=1e-12, abs=1e-300)

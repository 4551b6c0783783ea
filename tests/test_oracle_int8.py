"""Pins of the int8 oracle: codes against exact rationals, the product against
Python integers, the weight order against its index formula."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import codecs, int8


def _rint(x):
    """Nearest integer of a Fraction, ties to even."""
    low = x.numerator // x.denominator
    part = x - low
    half = Fraction(1, 2)
    return low + (1 if part > half or (part == half and low % 2) else 0)


def _row(kind, n, seed):
    g = np.random.default_rng(seed)
    if kind == "normal":
        return g.standard_normal(n).astype(np.float32)
    if kind == "bf16":
        return codecs.decode_bf16(codecs.round_to_bf16(g.standard_normal(n) * 8)).astype(np.float32)
    if kind == "ties":          # a scale of one: halves are ties
        return np.concatenate([[127.0], g.integers(-253, 254, n - 1) / 2]).astype(np.float32)
    if kind == "tiny":          # at the floor of the scale
        return (g.integers(-300, 300, n) * 2.0 ** -130).astype(np.float32)
    return (g.standard_normal(n) * 1e37).astype(np.float32)


@pytest.mark.parametrize("kind", ["normal", "bf16", "ties", "tiny", "huge"])
def test_quant_rows_against_rationals(kind):
    h = np.stack([_row(kind, 97, i) for i in range(6)])
    q, s = int8.quant_rows(h)
    for r in range(6):
        amax = max(abs(Fraction(float(v))) for v in h[r])
        sf = Fraction(float(s[r]))
        if s[r] > np.float32(int8.MIN_SCALE):     # correctly rounded: no neighbour is nearer
            for other in (np.nextafter(s[r], np.float32(0)), np.nextafter(s[r], np.float32(np.inf))):
                assert abs(amax / 127 - sf) <= abs(amax / 127 - Fraction(float(other)))
        else:
            assert amax / 127 <= sf
        assert [int(v) for v in q[r]] == [_rint(Fraction(float(v)) / sf) for v in h[r]]


def test_quant_rows_not_finite_and_zero():
    h = np.zeros((4, 8))
    h[1, 3], h[2, 4] = np.inf, np.nan
    h[3, 0] = -5.0
    q, s = int8.quant_rows(h)
    assert not q[:3].any() and q[3, 0] == -127
    assert s[0] == np.float32(2.0 ** -126) and np.isnan(s[1]) and np.isnan(s[2])


def test_norm_against_rationals():
    g = np.random.default_rng(3)
    y, r, w = (codecs.round_to_bf16(g.standard_normal((2, 16)) * 3), codecs.round_to_bf16(g.standard_normal((2, 16))),
               codecs.round_to_bf16(g.standard_normal(16) * .1))
    for offset in (0.0, 1.0):
        h, rb = int8.add_rms(y, r, w, 1e-6, offset)
        for i in range(2):
            v = [Fraction(float(a)) + Fraction(float(b)) for a, b in zip(codecs.decode_bf16(y[i]), codecs.decode_bf16(r[i]))]
            assert [int(x) for x in codecs.round_to_bf16(np.array([float(x) for x in v]))] == [int(x) for x in rb[i]]
            rv = [Fraction(float(x)) for x in codecs.decode_bf16(rb[i])]
            ms = sum(x * x for x in rv) / 16 + Fraction(float(np.float32(1e-6)))
            for x, gm, got in zip(rv, codecs.decode_bf16(w), h[i]):
                want = float(x) * (offset + float(gm)) / float(ms) ** 0.5
                assert abs(float(got) - want) <= 2.0 ** -24 * abs(want) * 1.0001


def test_silu_and_dequant():
    gu = codecs.round_to_bf16(np.array([[0.0, 1.0, -2.0, 80.0, 3.0, 2.0, 0.5, 1.0]]))
    h = int8.silu_mul(gu)
    want = [0.0, 2 / (1 + np.exp(-1.0)), -1 / (1 + np.exp(2.0)), 80.0]
    assert np.allclose(h[0], want, rtol=2.0 ** -23, atol=0)
    q, s = np.array([[127, -3, 0, 77]], np.int8), np.array([np.float32(1.2345678e-3)])
    d = codecs.decode_bf16(int8.dequant(q, s))
    for c, v in zip(q[0], d[0]):
        exact = Fraction(int(c)) * Fraction(float(s[0]))
        assert abs(Fraction(float(v)) - exact) <= abs(exact) / 256


def test_product_and_gemm_against_integers():
    g = np.random.default_rng(5)
    a, w = g.integers(-128, 128, (3, 80)).astype(np.int8), g.integers(-128, 128, (5, 80)).astype(np.int8)
    sa, sw = g.random(3).astype(np.float32), g.random(5).astype(np.float32)
    acc, c = int8.product(a, w), codecs.decode_bf16(int8.gemm(a, sa, w, sw))
    for m in range(3):
        for n in range(5):
            want = sum(int(x) * int(y) for x, y in zip(a[m], w[n]))
            assert acc[m, n] == want
            exact = want * Fraction(float(sa[m])) * Fraction(float(sw[n]))
            assert abs(Fraction(float(c[m, n])) - exact) <= abs(exact) * (Fraction(1, 256) + Fraction(4, 2 ** 24))


def test_prelayout_order():
    g = np.random.default_rng(6)
    for N, K in ((16, 64), (21, 80), (1, 16), (33, 256)):
        w = g.integers(-128, 128, (N, K)).astype(np.int8)
        out = int8.prelayout(w).view(np.int8)
        ks = -(-K // 128) * 2
        assert out.size == -(-N // 16) * ks * 1024
        for i in g.integers(0, out.size, 500):
            block, lane, byte = i // 1024, i % 1024 // 16, i % 16
            n, k = block // ks * 16 + lane % 16, block % ks * 64 + lane // 16 * 16 + byte
            assert out[i] == (w[n, k] if n < N and k < K else 0)

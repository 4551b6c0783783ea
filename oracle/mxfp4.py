"""MXFP4 quantisation, the W4A4 product and the mixture-of-experts routing,
written out from their definitions.

Test infrastructure (see the package docstring); never used by the product path.

Quantisation is the OCP microscaling rule for e2m1 with e8m0 scales: the shared
exponent is floor(log2(max |x|)) minus 2 (the exponent of e2m1's largest
binade), clamped to e8m0's range, and the elements are x / 2^e rounded to
nearest even with magnitudes beyond 6 saturated.  Readings: a block with an
infinity or NaN gets the scale byte 255 and zero codes; an all-zero block the
byte 0.
"""
import numpy as np

from .codecs import _floor_log2, decode_bf16
from .gemm import MX_BLOCK, dequant_mxfp4


def encode_e2m1(t):
    """Finite fp64 -> e2m1 codes, nearest even, saturating; the sign is kept on zeros."""
    t = np.asarray(t, np.float64)
    a = np.abs(t)
    quantum = np.exp2(np.clip(_floor_log2(np.where(a > 0, a, 1.0)), 0, 2) - 1.0)
    r = np.minimum(np.rint(a / quantum) * quantum, 6.0)
    code = np.searchsorted(np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]), r).astype(np.uint8)
    return np.where(np.signbit(t), code | 8, code).astype(np.uint8)


def quant_mxfp4(x):
    """fp64 rows [M, K] -> (packed codes uint8 [M, K/2], e8m0 bytes [M, K/32])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    b = x.reshape(M, K // MX_BLOCK, MX_BLOCK)
    finite = np.isfinite(b).all(axis=2)
    bf = np.where(finite[:, :, None], b, 0.0)
    amax = np.abs(bf).max(axis=2)
    e = np.where(amax > 0, _floor_log2(np.where(amax > 0, amax, 1.0)) - 2, -127)
    e = np.clip(e, -127, 127)
    codes = encode_e2m1(bf / np.exp2(e.astype(np.float64))[:, :, None])
    codes = np.where(finite[:, :, None], codes, 0).reshape(M, K).astype(np.uint8)
    scale = np.where(finite, e + 127, 255).astype(np.uint8)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), scale


def silu_mul(gu_bits):
    """bf16 [M, 2N] -> h = g * sigmoid(g) * u rounded once to fp32 (as fp64)."""
    gu = decode_bf16(gu_bits)
    N = gu.shape[1] // 2
    with np.errstate(over="ignore", invalid="ignore"):
        h = gu[:, :N] / (1.0 + np.exp(-gu[:, :N])) * gu[:, N:]
        return h.astype(np.float32).astype(np.float64)


def w4a4_gemm(a_packed, a_e8m0, w_packed, w_e8m0):
    """(c_exact, abs_sum) of C = A . W^T, both operands MXFP4."""
    A = dequant_mxfp4(a_packed, a_e8m0)
    W = dequant_mxfp4(w_packed, w_e8m0)
    return A @ W.T, np.abs(A) @ np.abs(W).T


def gemm_bound(c_exact, abs_sum, K):
    """How far the fp32-accumulated, bf16-rounded product may be off.  Each of
    the K/32 blocks of exact products is added into a running sum that never
    exceeds abs_sum, at the cost of at most one fp32 step (2^-23 relative; the
    adder may truncate): d = K/32 * 2^-23 * abs_sum.  The sum, at most
    |c| + d, is then rounded to bf16: half a step, 2^-8 relative, or half the
    smallest subnormal's step, 2^-134."""
    d = (K / 32.0) * 2.0 ** -23 * np.asarray(abs_sum, np.float64)
    return d + 2.0 ** -8 * (np.abs(c_exact) + d) + 2.0 ** -134


def assert_w4a4_close(c_bits, c_exact, abs_sum, K, what=""):
    got = decode_bf16(c_bits)
    off = np.abs(got - c_exact)
    bad = ~(off <= gemm_bound(c_exact, abs_sum, K))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at "
                           f"{np.argwhere(bad)[:3].tolist()}: got {got[bad][:3]}, want {c_exact[bad][:3]}")


def moe_sort(ids, E):
    """(rows, pos, offsets) of the kept pairs sorted by (id, pair)."""
    T, k = ids.shape
    flat = [int(v) for v in np.asarray(ids).reshape(-1)]
    rows = np.full(T * k, -1, np.int32)
    pos = np.full(T * k, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    lists = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(p)
    s = 0
    for e, pairs in enumerate(lists):
        for p in pairs:
            rows[s], pos[p] = p // k, s
            s += 1
        offsets[e + 1] = s
    return rows, pos.reshape(T, k), offsets


def moe_combine(y, pos, weights):
    """out[t] = sum_j weights[t, j] y[pos[t, j]], fp64, and the sum of magnitudes."""
    T, k = pos.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * y[pos[t, j]]
                mag[t] += np.abs(w * y[pos[t, j]])
    return out, mag


def moe_combine_backward(dout, y, pos, weights):
    """(dy, dweights, sum of the magnitudes of dweights' terms); dy rows that no pair names are NaN."""
    T, k = pos.shape
    dy = np.full(y.shape, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            s = pos[t, j]
            if s >= 0:
                dy[s] = float(weights[t, j]) * dout[t]
                dw[t, j] = (dout[t] * y[s]).sum()
                mag[t, j] = np.abs(dout[t] * y[s]).sum()
    return dy, dw, mag

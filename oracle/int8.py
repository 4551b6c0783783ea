"""int8 quantisation with one scale per row, its producers and the W8A8 product,
written out from their definitions.

Test infrastructure (see the package docstring); never used by the product path.

A row h of fp32 values is quantised to s = max(fp32(max |h| / 127), 2^-126) and
q = h / s rounded to nearest even.  Reading: a row with an infinity or a NaN gets
a NaN scale and zero codes.
"""
import numpy as np

from .codecs import bf16_ulp, decode_bf16, round_to_bf16  # noqa: F401

MIN_SCALE = 2.0 ** -126


def quant_rows(h):
    """fp64 rows that hold fp32 values -> (int8 codes [M, K], fp32 scales [M]).
    fp64 quotients of fp32 values round as the exact ones do: a quotient that is
    no half-integer is at least 2^-26 away from one."""
    h = np.asarray(h, np.float64)
    finite = np.isfinite(h).all(axis=1)
    hf = np.where(finite[:, None], h, 0.0)
    s = np.maximum((np.abs(hf).max(axis=1) / 127.0).astype(np.float32), np.float32(MIN_SCALE))
    q = np.rint(hf / s.astype(np.float64)[:, None])
    assert np.abs(q).max(initial=0.0) <= 127
    return q.astype(np.int8), np.where(finite, s, np.float32("nan")).astype(np.float32)


def add_rms(y_bits, r_bits, g_bits, eps, offset):
    """(h as fp32, residual_out bits): r = bf16(y + residual), h = fp32 of the real
    r / sqrt(mean r^2 + eps) * (offset + gamma)."""
    with np.errstate(all="ignore"):
        y = decode_bf16(y_bits)
        rb = np.asarray(y_bits, np.uint16) if r_bits is None else round_to_bf16(y + decode_bf16(r_bits))
        r = decode_bf16(rb)
        inv = 1.0 / np.sqrt((r * r).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
        h = r * inv * (np.float64(np.float32(offset)) + decode_bf16(g_bits))
        return h.astype(np.float32), rb


def silu_mul(gu_bits):
    """bf16 [M, 2N] -> fp32 of g / (1 + exp(-g)) * u."""
    gu = decode_bf16(gu_bits)
    n = gu.shape[1] // 2
    g, u = gu[:, :n], gu[:, n:]
    with np.errstate(all="ignore"):
        return (g / (1.0 + np.exp(-g)) * u).astype(np.float32)


def dequant(q, s):
    """bf16 bits of q * s, rounded once."""
    with np.errstate(all="ignore"):
        return round_to_bf16(np.asarray(q, np.float64) * np.asarray(s, np.float64)[:, None])


def product(a, w):
    """sum_k a[m,k] w[n,k], whole numbers (exact in fp64: K < 2^17)."""
    return np.asarray(a, np.float64) @ np.asarray(w, np.float64).T


def gemm(a, a_scale, w, w_scale):
    """bf16 bits of fp32(fp32(fp32(sum) * a_scale) * w_scale), the entry point's order."""
    with np.errstate(all="ignore"):
        acc = product(a, w).astype(np.float32)
        c = acc * np.asarray(a_scale, np.float32)[:, None] * np.asarray(w_scale, np.float32)[None, :]
        return round_to_bf16(c.astype(np.float64))


def prelayout(w):
    """int8 [N, K] -> the bytes of the fragment order, rows padded to 16 and K to 128 with zeros."""
    N, K = w.shape
    nt, ks = (N + 15) // 16, (K + 127) // 128 * 2
    full = np.zeros((nt * 16, ks * 64), np.int8)
    full[:N, :K] = w
    # [tile, row, step, chunk, byte] -> [tile, step, chunk, row, byte]
    return full.reshape(nt, 16, ks, 4, 16).transpose(0, 2, 3, 1, 4).reshape(-1).view(np.uint8)

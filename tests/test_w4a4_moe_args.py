"""Refusals of the MXFP4 W4A4 and mixture-of-experts entry points, in the C ABI
and in the Python binding.  CPU only: every call is refused before any device
memory is touched."""
import ctypes

import pytest
import torch

import block_scaled_precision_04_amd as bs
from block_scaled_precision_04_amd import _binding
from block_scaled_precision_04_amd._binding import WDesc, BS_WDESC_MAGIC, BS_LAYOUT_FP8_BLOCK, BS_LAYOUT_MXFP4

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
N, K = 256, 512


@pytest.fixture(scope="module")
def blib():
    import os
    if not os.path.exists(_binding.LIB_PATH):
        from block_scaled_precision_04_amd import build
        build.build()
    return _binding.lib()


def _mx(n=N, k=K):
    codes, sc = n * k // 2, n // 16 * ((k // 128 + 3) // 4) * 256
    return WDesc(BS_WDESC_MAGIC, BS_LAYOUT_MXFP4, n, k, codes, codes, sc, codes + sc)


def test_w4a4_refusals(blib):
    def call(M=8, n=N, k=K, a=FAKE, lda=None, s=FAKE, lds=None, d=None, w=FAKE, c=FAKE, ldc=None, ws=None, wsn=0):
        d = _mx(n, k) if d is None else d
        return blib.bsgemm_w4a4_mxfp4(a, k // 2 if lda is None else lda, s, k // 32 if lds is None else lds,
                                      ctypes.byref(d), w, c, n if ldc is None else ldc, M, n, k, ws, wsn, None)
    assert call(M=0, a=None, s=None, w=None, c=None) == 0
    assert call(a=None) == -1 and call(s=None) == -1 and call(w=None) == -1 and call(c=None) == -1
    assert call(M=-1) == -2 and call(M=(1 << 22) + 1) == -2
    assert call(n=200, d=_mx()) == -2 and call(k=576, d=_mx()) == -2 and call(n=0, d=_mx()) == -2
    assert call(n=240, d=_mx()) == -4                       # a descriptor of another shape
    assert call(d=WDesc(BS_WDESC_MAGIC, BS_LAYOUT_FP8_BLOCK, N, K, N * K, 0, 0, N * K)) == -4
    assert call(lda=K // 2 - 16) == -3 and call(lda=K // 2 + 8) == -3
    assert call(lds=K // 32 - 4) == -3 and call(lds=K // 32 + 2) == -3
    assert call(ldc=N - 4) == -3 and call(ldc=N + 2) == -3
    assert call(a=ODD) == -3 and call(s=ODD) == -3 and call(w=ctypes.c_void_p(0x10080)) == -3 and call(c=ODD) == -3
    assert call(M=1 << 20, lda=1 << 12) == -2               # M * lda = 2^32
    assert call(M=1 << 20, lds=1 << 12) == -2
    assert call(lda=-16) == -3 and call(lds=1 << 40) == -2
    # a K split needs its workspace
    need = bs.workspace_bytes(bs.BS_OP_W4A4_MXFP4, 8, 256, 17408)
    assert need > 64 * 1024
    assert call(k=17408) == -5 and call(k=17408, ws=FAKE, wsn=need - 1) == -5
    assert call(k=17408, ws=ctypes.c_void_p(0x10080), wsn=need) == -3
    assert bs.workspace_bytes(bs.BS_OP_W4A4_MXFP4, 8, 250, 512) == 0
    assert bs.workspace_bytes(bs.BS_OP_W4A4_MXFP4, 8192, 10240, 5120) == 0


def test_grouped_refusals(blib):
    def call(S=8, E=4, Ma=8, n=N, k=K, a=FAKE, lda=None, s=FAKE, lds=None, off=FAKE, rows=None, d=None, w=FAKE,
             stride=None, c=FAKE, ldc=None):
        d = _mx(n, k) if d is None else d
        return blib.bsgemm_w4a4_mxfp4_grouped(a, k // 2 if lda is None else lda, s, k // 32 if lds is None else lds, Ma,
                                              off, rows, ctypes.byref(d), w, d.total_bytes if stride is None else stride,
                                              c, n if ldc is None else ldc, S, E, n, k, None)
    assert call(S=0, a=None, off=None, w=None, c=None) == 0
    assert call(a=None) == -1 and call(s=None) == -1 and call(off=None) == -1 and call(w=None) == -1
    assert call(c=None) == -1
    assert call(S=-1) == -2 and call(S=(1 << 24) + 1) == -2 and call(Ma=0) == -2
    assert call(E=0) == -2 and call(E=1025) == -2 and call(n=200, d=_mx()) == -2 and call(k=64, d=_mx()) == -2
    assert call(stride=_mx().total_bytes - 256) == -4 and call(stride=_mx().total_bytes + 16) == -4
    assert call(d=WDesc(0, BS_LAYOUT_MXFP4, N, K, 0, 0, 0, 0), stride=1 << 20) == -4
    assert call(off=ODD) == -3 and call(rows=ODD) == -3 and call(lda=K // 2 + 4) == -3 and call(lds=K // 32 + 1) == -3
    assert call(Ma=1 << 24) == -2                           # Ma * lda = 2^32


def test_quantiser_refusals(blib):
    q = blib.quant_mxfp4
    assert q(None, 0, None, None, 0, 64, None) == 0
    assert q(None, 64, FAKE, FAKE, 4, 64, None) == -1 and q(FAKE, 64, FAKE, None, 4, 64, None) == -1
    assert q(FAKE, 64, FAKE, FAKE, 4, 48, None) == -2 and q(FAKE, 64, FAKE, FAKE, -4, 64, None) == -2
    assert q(FAKE, 1 << 14, FAKE, FAKE, 1 << 20, 1 << 14, None) == -2      # 2^31 chunks
    assert q(FAKE, 56, FAKE, FAKE, 4, 64, None) == -3 and q(FAKE, 68, FAKE, FAKE, 4, 64, None) == -3
    assert q(ctypes.c_void_p(0x10008), 64, FAKE, FAKE, 4, 64, None) == -3 and q(FAKE, 64, ODD, FAKE, 4, 64, None) == -3
    s = blib.silu_mul_quant_mxfp4
    assert s(None, None, None, None, 0, 64, None) == 0
    assert s(None, FAKE, FAKE, None, 4, 64, None) == -1 and s(FAKE, FAKE, FAKE, None, 4, 40, None) == -2
    assert s(ODD, FAKE, FAKE, None, 4, 64, None) == -3 and s(FAKE, FAKE, FAKE, ODD, 4, 64, None) == -3
    d = blib.dequant_mxfp4
    assert d(None, None, None, 0, 64, None) == 0
    assert d(FAKE, FAKE, None, 4, 64, None) == -1 and d(FAKE, FAKE, FAKE, 4, 16, None) == -2
    assert d(FAKE, FAKE, ctypes.c_void_p(0x10008), 4, 64, None) == -3 and d(ODD, FAKE, FAKE, 4, 64, None) == -3


def test_moe_refusals(blib):
    s = blib.moe_sort
    assert s(FAKE, FAKE, FAKE, None, 4, 2, 8, None, 0, None) == -1 and s(None, FAKE, FAKE, FAKE, 4, 2, 8, None, 0, None) == -1
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 0, 8, None, 0, None) == -2 and s(FAKE, FAKE, FAKE, FAKE, 4, 2, 0, None, 0, None) == -2
    assert s(FAKE, FAKE, FAKE, FAKE, 4, 2, 1025, None, 0, None) == -2 and s(FAKE, FAKE, FAKE, FAKE, -1, 2, 8, None, 0, None) == -2
    assert s(FAKE, FAKE, FAKE, FAKE, 1 << 22, 5, 8, None, 0, None) == -2
    assert s(ODD, FAKE, FAKE, FAKE, 4, 2, 8, None, 0, None) == -3
    need = bs.workspace_bytes(bs.BS_OP_MOE_SORT, 5000, 2, 8)
    assert need > 64 * 1024 and bs.workspace_bytes(bs.BS_OP_MOE_SORT, 2048, 2, 8) == 0
    assert s(FAKE, FAKE, FAKE, FAKE, 5000, 2, 8, None, 0, None) == -5
    assert s(FAKE, FAKE, FAKE, FAKE, 5000, 2, 8, FAKE, need - 1, None) == -5
    assert s(FAKE, FAKE, FAKE, FAKE, 5000, 2, 8, ctypes.c_void_p(0x10040), need, None) == -3
    for fn, args in ((blib.moe_gather, 3), (blib.moe_combine, 4), (blib.moe_combine_backward, 6)):
        assert fn(*[None] * args, 0, 2, 64, None) == 0
        assert fn(*[None] * args, 4, 2, 64, None) == -1
        ok = [FAKE] * args
        assert fn(*ok, 4, 2, 60, None) == -2 and fn(*ok, 4, 2, 32776, None) == -2 and fn(*ok, 4, 0, 64, None) == -2
        assert fn(*ok, 1 << 22, 8, 64, None) == -2 and fn(*ok, -1, 2, 64, None) == -2
        for i in range(args):
            bad = list(ok)
            bad[i] = ODD
            assert fn(*bad, 4, 2, 64, None) == -3, (fn, i)


def _refused(fn, match, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_refusals():
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    a, s = torch.zeros((8, K // 2), dtype=u8), torch.zeros((8, K // 32), dtype=u8)
    d = _mx()
    w = torch.zeros(d.total_bytes, dtype=u8)
    g = bs.bsgemm_w4a4_mxfp4
    _refused(g, "descriptor K", a[:, :64], s, d, w)
    _refused(g, "a_scale has shape", a, s[:, :8], d, w)
    _refused(g, "a has dtype", a.to(torch.int16), s, d, w)
    _refused(g, "unit stride", torch.zeros((K // 2, 8), dtype=u8).t(), s, d, w)
    _refused(g, "the layout needs", a, s, d, w[:-1])
    _refused(g, "out has shape", a, s, d, w, out=torch.zeros((8, N + 16), dtype=bf))
    _refused(g, "out has dtype", a, s, d, w, out=torch.zeros((8, N)))
    _refused(g, "on a GPU", a, s, d, w)
    gg = bs.bsgemm_w4a4_mxfp4_grouped
    we, off = torch.zeros((4, d.total_bytes), dtype=u8), torch.zeros(5, dtype=i32)
    _refused(gg, "offsets has shape", a, s, off[:4], d, we)
    _refused(gg, "offsets has dtype", a, s, off.long(), d, we)
    _refused(gg, "w_pre must be a 2-D", a, s, off, d, w)
    _refused(gg, "the layout needs", a, s, off, d, we[:, :-256])
    _refused(gg, "rows has dtype", a, s, off, d, we, rows=torch.zeros(8, dtype=torch.int64))
    _refused(gg, "out has shape", a, s, off, d, we, rows=torch.zeros(9, dtype=i32), out=torch.zeros((8, N), dtype=bf))
    _refused(gg, "on a GPU", a, s, off, d, we)
    x = torch.zeros((4, 64), dtype=bf)
    _refused(bs.quant_mxfp4, "multiple of 32", x[:, :48])
    _refused(bs.quant_mxfp4, "x has dtype", x.float())
    _refused(bs.quant_mxfp4, "q has shape", x, q=torch.zeros((4, 64), dtype=u8))
    _refused(bs.quant_mxfp4, "on a GPU", x)
    _refused(bs.silu_mul_quant_mxfp4, "multiple of 32", x[:, :48])
    _refused(bs.silu_mul_quant_mxfp4, "rows has shape", x, rows=torch.zeros(2, dtype=i32))
    _refused(bs.silu_mul_quant_mxfp4, "on a GPU", x)
    _refused(bs.dequant_mxfp4, "scale has shape", torch.zeros((4, 32), dtype=u8), torch.zeros((4, 1), dtype=u8))
    _refused(bs.dequant_mxfp4, "on a GPU", torch.zeros((4, 32), dtype=u8), torch.zeros((4, 2), dtype=u8))
    ids = torch.zeros((4, 2), dtype=i32)
    _refused(bs.moe_sort, "ids has dtype", ids.long(), 8)
    _refused(bs.moe_sort, "pos has shape", ids, 8, pos=torch.zeros((2, 4), dtype=i32))
    _refused(bs.moe_sort, "positive int", ids, -1)
    _refused(bs.moe_sort, "positive int", ids, 8.0)
    _refused(bs.moe_sort, "on a GPU", ids, 8)
    y = torch.zeros((8, 64), dtype=bf)
    _refused(bs.moe_gather, "x has shape", y, ids)
    _refused(bs.moe_gather, "out has shape", x, ids, out=x)
    _refused(bs.moe_combine, "y has shape", x, ids)
    _refused(bs.moe_combine, "weights has dtype", y, ids, weights=torch.zeros((4, 2), dtype=bf))
    _refused(bs.moe_combine, "pos must be contiguous", y, torch.zeros((2, 4), dtype=i32).t())
    _refused(bs.moe_combine, "on a GPU", y, ids)
    _refused(bs.moe_combine_backward, "weights is required", x, y, ids, None)
    _refused(bs.moe_combine_backward, "dweights has shape", x, y, ids, torch.zeros((4, 2)), dweights=torch.zeros(8))
    _refused(bs.moe_combine_backward, "on a GPU", x, y, ids, torch.zeros((4, 2)))
    _refused(bs.prelayout_mxfp4_experts, "3-D", w, w)
    _refused(bs.prelayout_mxfp4_experts, "w_e8m0 has shape", torch.zeros((2, 16, 64), dtype=u8), torch.zeros((2, 16, 2), dtype=u8))

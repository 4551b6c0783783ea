"""W4A4 MXFP4 GEMM, dense and grouped, against the fp64 oracle, and the whole
mixture-of-experts layer that the operators make together."""
import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from block_scaled_precision_04_amd import synth
from oracle import codecs, mxfp4
from tests.gpu_util import dev_bf16, dev_u8, host_bits16

pytestmark = pytest.mark.gpu


def _operand(g, M, K):
    """Uniform codes, scales over a few binades (the weight workload's distribution)."""
    return synth.uniform_bytes(g, (M, K // 2)), synth.uniform_exponents(g, (M, K // 32))


def _dense(M, N, K, seed=0):
    g = synth.rng(seed + M * 7 + N * 3 + K)
    a, ae = _operand(g, M, K)
    w, we = _operand(g, N, K)
    pre, desc = bs.prelayout_mxfp4(dev_u8(w), dev_u8(we))
    return a, ae, w, we, pre, desc


# every configuration of the weight stream and every tile shape, K with and
# without whole windows of 512 (the scale loads differ), ragged M and N
DENSE = [
    # weight stream, up to 16 rows: K = 512, 1024, 2048, 5120 (one run), longer (split)
    (1, 16, 128), (8, 10240, 512), (3, 48, 1024), (7, 272, 768), (5, 272, 1664), (16, 48, 2048), (1, 5120, 2304),
    (16, 48, 5120), (16, 96, 12544), (2, 16, 5248), (9, 4112, 2304), (12, 8208, 2304), (3, 4112, 12416),
    # weight stream, 17 to 64 rows of long K
    (20, 48, 12416), (33, 48, 12288), (64, 80, 12544),
    # 64 x 64 tiles: short K, longer K in two K groups
    (17, 160, 1152), (32, 256, 2048), (33, 144, 256), (64, 1040, 1280), (65, 16, 128), (65, 128, 1024),
    (100, 272, 2176), (128, 128, 128), (129, 400, 384), (300, 1296, 640), (513, 144, 8192), (200, 2064, 512),
    (1000, 528, 256), (65, 144, 12416), (65, 144, 12288), (70, 64, 16384),
    # 64 x 128 tiles
    (513, 2064, 1024), (513, 2064, 896), (600, 2064, 4224), (300, 4112, 2048),
    # 128 x 128 tiles
    (1100, 2064, 1024), (1100, 2064, 1152),
    # 128 x 256 tiles
    (1000, 4112, 640), (900, 4112, 1024),
]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    a, ae, w, we, pre, desc = _dense(M, N, K)
    ws = bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, M, N, K)
    c = bs.bsgemm_w4a4_mxfp4(dev_u8(a), dev_u8(ae), desc, pre, ws=ws)
    torch.cuda.synchronize()
    ce, asum = mxfp4.w4a4_gemm(a, ae, w, we)
    mxfp4.assert_w4a4_close(host_bits16(c), ce, asum, K, f"M={M} N={N} K={K}")
    if ws is not None:                     # the counters are left ready, and a second call agrees
        assert not ws[: 64 * 1024].any()
        c2 = bs.bsgemm_w4a4_mxfp4(dev_u8(a), dev_u8(ae), desc, pre, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(c, c2)


@pytest.mark.parametrize("M,N,K", [
    (4096, 4096, 1024), (3000, 5136, 512), (3333, 5136, 640), (2048, 10240, 256), (4352, 4240, 2048),  # 128 x 256
    (1025, 10256, 2048), (1025, 10256, 2176),    # 256 x 256
    (4352, 4240, 2176), (2048, 9008, 2048),      # 256 x 256 over whole rounds, the last columns smaller tiles
])
def test_dense_large_sampled(M, N, K):
    a, ae, w, we, pre, desc = _dense(M, N, K)
    c = bs.bsgemm_w4a4_mxfp4(dev_u8(a), dev_u8(ae), desc, pre, ws=bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, M, N, K))
    torch.cuda.synchronize()
    got = host_bits16(c)
    # whole rows of the first, last and some tiles
    rows = np.unique(np.concatenate([[0, 1, 31, 32, 127, 128, 255, 256, M - 1], np.arange(5, M, 251)]))
    ce, asum = mxfp4.w4a4_gemm(a[rows], ae[rows], w, we)
    mxfp4.assert_w4a4_close(got[rows], ce, asum, K, f"M={M} N={N} K={K}")


@pytest.mark.parametrize("K", [640, 512])
@pytest.mark.parametrize("M", [3, 40, 130])
def test_dense_strides_and_guard(M, K):
    """Padded activation, scale and output rows; the padding keeps what it held."""
    N = 272
    a, ae, w, we, pre, desc = _dense(M, N, K, 1)
    abuf = torch.full((M, K // 2 + 48), 0x77, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((M, K // 32 + 4), 0xFF, dtype=torch.uint8, device="cuda")   # NaN scales beside the used ones
    abuf[:, : K // 2] = dev_u8(a)
    sbuf[:, : K // 32] = dev_u8(ae)
    for ldc in (N + 4, N + 8):
        out = torch.full((M + 2, ldc), 7.0, dtype=torch.bfloat16, device="cuda")
        bs.bsgemm_w4a4_mxfp4(abuf[:, : K // 2], sbuf[:, : K // 32], desc, pre, out=out[:M, :N],
                             ws=bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, M, N, K))
        torch.cuda.synchronize()
        ce, asum = mxfp4.w4a4_gemm(a, ae, w, we)
        mxfp4.assert_w4a4_close(host_bits16(out[:M, :N].contiguous()), ce, asum, K)
        assert (out[M:] == 7).all() and (out[:M, N:] == 7).all()


@pytest.mark.parametrize("M", [2, 70])
def test_dense_scale_ends_and_nan(M):
    """Scales at both ends of e8m0 (their products stay inside fp32), and the NaN scale."""
    N, K = 64, 256
    a, ae, w, we, _, _ = _dense(M, N, K, 2)
    ae[0], we[:] = 0, 254
    ae[1:] = 60
    ae[1, 3] = 255
    pre, desc = bs.prelayout_mxfp4(dev_u8(w), dev_u8(we))
    c = bs.bsgemm_w4a4_mxfp4(dev_u8(a), dev_u8(ae), desc, pre, ws=bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, M, N, K))
    torch.cuda.synchronize()
    got = host_bits16(c)
    keep = np.arange(M) != 1
    ce, asum = mxfp4.w4a4_gemm(a[keep], ae[keep], w, we)
    mxfp4.assert_w4a4_close(got[keep], ce, asum, K)
    assert np.isnan(codecs.decode_bf16(got[1])).all()


def test_quantised_linear_both_activation_forms():
    """quant_mxfp4 of activations and weights feeds the product as it stands."""
    M, N, K = 70, 96, 256
    g = synth.rng(3)
    x, wt = synth.bf16_normal(g, (M, K), 1.0, outlier_p=0.01), synth.bf16_normal(g, (N, K), 0.02)
    q, s = bs.quant_mxfp4(dev_bf16(x))
    pre, desc = bs.prelayout_mxfp4(*bs.quant_mxfp4(dev_bf16(wt)))
    c = bs.bsgemm_w4a4_mxfp4(q, s, desc, pre, ws=bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, M, N, K))
    torch.cuda.synchronize()
    ce, asum = mxfp4.w4a4_gemm(*mxfp4.quant_mxfp4(codecs.decode_bf16(x)), *mxfp4.quant_mxfp4(codecs.decode_bf16(wt)))
    mxfp4.assert_w4a4_close(host_bits16(c), ce, asum, K)


# --------------------------------------------------------------------- grouped
def _experts(g, E, N, K):
    w, we = synth.uniform_bytes(g, (E, N, K // 2)), synth.uniform_exponents(g, (E, N, K // 32))
    pre, desc = bs.prelayout_mxfp4_experts(dev_u8(w), dev_u8(we))
    return w, we, pre, desc


def _grouped(counts, N, K, Ma, tail=0, seed=0, with_rows=True):
    E = len(counts)
    n = int(sum(counts))
    S = n + tail
    g = synth.rng(seed + N + K + S)
    Ma = Ma if with_rows else S
    a, ae = _operand(g, Ma, K)
    w, we, pre, desc = _experts(g, E, N, K)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = g.integers(0, Ma, S).astype(np.int32)
    rows[n:] = -1
    out = torch.full((S, N), 7.0, dtype=torch.bfloat16, device="cuda")
    bs.bsgemm_w4a4_mxfp4_grouped(dev_u8(a), dev_u8(ae), torch.from_numpy(off).cuda(), desc, pre,
                                 rows=torch.from_numpy(rows).cuda() if with_rows else None, out=out)
    torch.cuda.synchronize()
    got = host_bits16(out)
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        if len(r):
            src = rows[r] if with_rows else r
            ce, asum = mxfp4.w4a4_gemm(a[src], ae[src], w[e], we[e])
            mxfp4.assert_w4a4_close(got[r], ce, asum, K, f"expert {e} of {E}, {len(r)} rows")
    assert (got[n:] == 0x40E0).all()


GROUPED = [([1], 16, 128, 1), ([0, 1, 0], 48, 384, 3), ([3, 0, 17, 1, 16], 144, 640, 9), ([1] * 9, 1024, 2048, 4),
           ([40, 0, 0, 1, 30, 33], 80, 256, 50), ([20] * 7 + [64, 65], 272, 1152, 100), ([129, 0, 128, 1, 300], 144, 384, 77),
           ([500, 3, 0, 0], 400, 512, 333), ([0, 0, 90], 128, 2176, 90), ([60] * 5, 16, 128, 11)]


@pytest.mark.parametrize("counts,N,K,Ma", GROUPED)
def test_grouped(counts, N, K, Ma):
    _grouped(counts, N, K, Ma)
    _grouped(counts, N, K, Ma, tail=13, seed=1)
    _grouped(counts, N, K, Ma, seed=2, with_rows=False)


@pytest.mark.parametrize("E,N,K", [
    (3, 80, 2304),     # few workgroups: four K groups, the second run of K steps partly idle
    (4, 144, 896),     # two K groups that cover all of K
    (70, 272, 2176),   # two K groups, runs of 8 steps, one in the last
    (70, 1040, 1152),  # no K groups, runs of 4 steps
    (70, 48, 384)])
def test_grouped_few_rows(E, N, K):
    """The weight stream's forms, at most 9 rows an expert on average, some with more."""
    g = np.random.default_rng(E + N)
    counts = np.where(g.random(E) < 0.8, g.integers(1, 5, E), 0)
    counts[E // 2] = 18
    _grouped(counts.tolist(), N, K, 11)
    _grouped(counts.tolist(), N, K, 5, tail=3, seed=1)


@pytest.mark.parametrize("counts,N,K", [([20] * 6 + [64, 1], 272, 2048), ([25, 0, 31, 12], 144, 1664),
                                        ([65, 0, 0, 1, 30, 33], 80, 4096), ([20] * 6 + [64, 1], 272, 512),
                                        ([25, 17, 31, 12], 400, 896)])
def test_grouped_some_rows(counts, N, K):
    """Between 10 and 32 rows an expert: 64 x 128 tiles for long K, 128 x 256 for short."""
    _grouped(counts, N, K, 50)
    _grouped(counts, N, K, 50, tail=5, seed=1)


@pytest.mark.parametrize("N,K", [(80, 256), (528, 384), (2048, 128)])
def test_grouped_many_row_tiles(N, K):
    """Enough row tiles that runs of them go to one XCD, with a rest that does not."""
    counts = [300, 129, 0, 512, 257, 1, 640, 128, 127, 400, 0, 383, 5, 700]
    _grouped(counts, N, K, 222)
    _grouped(counts, N, K, 222, tail=200, seed=1)


def test_grouped_many_experts():
    """More experts than one pass of the tile search covers, most of them empty."""
    g = np.random.default_rng(6)
    counts = np.where(g.random(700) < 0.1, g.integers(1, 20, 700), 0)
    _grouped(counts.tolist(), 32, 128, 21)
    counts[:] = 0
    counts[699] = 3
    _grouped(counts.tolist(), 32, 128, 5, tail=2)


@pytest.mark.parametrize("K", [256, 1152])
@pytest.mark.parametrize("per", [2, 20, 70])
def test_grouped_wrong_offsets_and_rows(per, K):
    """Offsets and rows out of range: nothing outside the S output rows is
    written, and the experts whose own slots and rows are in range are right."""
    E, N, Ma, S = 4, 48, 9, 4 * per
    g = synth.rng(per + K)
    a, ae = _operand(g, Ma, K)
    w, we, pre, desc = _experts(g, E, N, K)
    off = np.array([0, per, 2 * per, 2 * per, S + 1000000], np.int32)    # expert 3: clamped to S
    rows = g.integers(0, Ma, S).astype(np.int32)
    rows[per:2 * per] = g.choice([-7, -1, Ma, 1 << 30, -(1 << 31)], per)
    buf = torch.full((S + 40, N), 7.0, dtype=torch.bfloat16, device="cuda")
    bs.bsgemm_w4a4_mxfp4_grouped(dev_u8(a), dev_u8(ae), torch.from_numpy(off).cuda(), desc, pre,
                                 rows=torch.from_numpy(rows).cuda(), out=buf[20:20 + S])
    torch.cuda.synchronize()
    got = host_bits16(buf)
    assert (got[:20] == 0x40E0).all() and (got[20 + S:] == 0x40E0).all()
    got = got[20:20 + S]
    for e, r in ((0, slice(0, per)), (3, slice(2 * per, S))):
        ce, asum = mxfp4.w4a4_gemm(a[rows[r]], ae[rows[r]], w[e], we[e])
        mxfp4.assert_w4a4_close(got[r], ce, asum, K, f"expert {e}")
    off[:] = [S + 5, -3, per, 0, -(1 << 31)]                              # decreasing, negative
    bs.bsgemm_w4a4_mxfp4_grouped(dev_u8(a), dev_u8(ae), torch.from_numpy(off).cuda(), desc, pre,
                                 rows=torch.from_numpy(rows).cuda(), out=buf[20:20 + S])
    torch.cuda.synchronize()
    got = host_bits16(buf)
    assert (got[:20] == 0x40E0).all() and (got[20 + S:] == 0x40E0).all()


def test_grouped_no_slots():
    g = synth.rng(1)
    _, _, pre, desc = _experts(g, 3, 16, 128)
    a, ae = _operand(g, 4, 128)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = bs.bsgemm_w4a4_mxfp4_grouped(dev_u8(a), dev_u8(ae), off, desc, pre,
                                       rows=torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 16)
    guard = torch.full((4, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    bs.bsgemm_w4a4_mxfp4_grouped(dev_u8(a), dev_u8(ae), off, desc, pre, out=guard)
    torch.cuda.synchronize()
    assert (guard == 7).all()


def test_grouped_padded_weights_and_outputs():
    """Expert weights further apart than their size, and padded output rows."""
    g = synth.rng(9)
    E, N, K, Ma = 3, 32, 256, 6
    w, we, pre, desc = _experts(g, E, N, K)
    wide = torch.zeros((E, pre.shape[1] + 512), dtype=torch.uint8, device="cuda")
    wide[:, : pre.shape[1]] = pre
    a, ae = _operand(g, Ma, K)
    off = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    out = torch.full((Ma, N + 4), 7.0, dtype=torch.bfloat16, device="cuda")
    bs.bsgemm_w4a4_mxfp4_grouped(dev_u8(a), dev_u8(ae), off, desc, wide[:, : pre.shape[1]], out=out[:, :N])
    torch.cuda.synchronize()
    got = host_bits16(out[:, :N].contiguous())
    for e, (r0, r1) in enumerate(((0, 2), (2, 2), (2, 6))):
        if r1 > r0:
            ce, asum = mxfp4.w4a4_gemm(a[r0:r1], ae[r0:r1], w[e], we[e])
            mxfp4.assert_w4a4_close(got[r0:r1], ce, asum, K)
    assert (out[:, N:] == 7).all()


# ------------------------------------------------------- the operators together
def _layer(x, gate, w1, w2, k, E, ws, bufs=None):
    """A mixture-of-experts MLP: gate (skinny bf16 GEMM), top-k, sort, quantise,
    experts' gate/up products, SiLU * up + quantise, experts' down products, combine."""
    logits = bs.gemm_bf16_skinny(x, gate, ws=ws["gate"])
    top, ids = torch.topk(logits.float(), k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    rows, pos, off = bs.moe_sort(ids.int(), E, ws=ws["sort"])
    q, s = bs.quant_mxfp4(x)
    h = bs.bsgemm_w4a4_mxfp4_grouped(q, s, off, w1[1], w1[0], rows=rows)
    hq, hs = bs.silu_mul_quant_mxfp4(h, rows=off[E:])
    y = bs.bsgemm_w4a4_mxfp4_grouped(hq, hs, off, w2[1], w2[0])
    return bs.moe_combine(y, pos, weights), ids, weights, h, y, pos


@pytest.mark.parametrize("T,k,E", [(1, 2, 16), (24, 4, 16), (64, 8, 16)])
def test_moe_layer(T, k, E):
    H, I = 256, 128
    g = synth.rng(T)
    x = synth.bf16_normal(g, (T, H), 1.0)
    gate = synth.bf16_normal(g, (E, H), 0.05)
    w1b, w2b = synth.bf16_normal(g, (E, 2 * I, H), 0.05), synth.bf16_normal(g, (E, H, I), 0.05)

    def experts(b):
        e, n, kk = b.shape
        q, s = bs.quant_mxfp4(dev_bf16(b.reshape(e * n, kk)))
        return bs.prelayout_mxfp4_experts(q.view(e, n, kk // 2), s.view(e, n, kk // 32))
    w1, w2 = experts(w1b), experts(w2b)
    ws = {"gate": bs.alloc_workspace(bs.BS_OP_BF16_SKINNY, T, E, H),
          "sort": bs.alloc_workspace(bs.BS_OP_MOE_SORT, T, k, E)}
    xd, gd = dev_bf16(x), dev_bf16(gate)
    out, ids, weights, h, y, pos = _layer(xd, gd, w1, w2, k, E, ws)
    torch.cuda.synchronize()
    # each stage against the oracle on the stage's own inputs
    ids_h, pos_h = ids.cpu().numpy(), pos.cpu().numpy()
    rows_o, pos_o, off_o = mxfp4.moe_sort(ids_h, E)
    assert np.array_equal(pos_h, pos_o)
    xq = mxfp4.quant_mxfp4(codecs.decode_bf16(x))
    hb, yb = host_bits16(h), host_bits16(y)
    hq = mxfp4.quant_mxfp4(mxfp4.silu_mul(hb))
    for e in range(E):
        r = np.arange(off_o[e], off_o[e + 1])
        if len(r) == 0:
            continue
        we1, we2 = (mxfp4.quant_mxfp4(codecs.decode_bf16(b[e])) for b in (w1b, w2b))
        ce, asum = mxfp4.w4a4_gemm(xq[0][rows_o[r]], xq[1][rows_o[r]], *we1)
        mxfp4.assert_w4a4_close(hb[r], ce, asum, H, f"gate/up of expert {e}")
        ce, asum = mxfp4.w4a4_gemm(hq[0][r], hq[1][r], *we2)
        mxfp4.assert_w4a4_close(yb[r], ce, asum, I, f"down of expert {e}")
    w = weights.cpu().numpy()
    want, mag = mxfp4.moe_combine(codecs.decode_bf16(yb), pos_h, w)
    d = 2 * k * 2.0 ** -24 * mag
    got = codecs.decode_bf16(host_bits16(out))
    assert (np.abs(got - want) <= d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -134).all()


def test_graph_replays_match_eager():
    """The routed layer and a split dense product captured once, replayed with new
    inputs and the program's own eager work between the replays."""
    T, k, E, H, I = 24, 4, 16, 256, 128
    g = synth.rng(77)
    w1 = _experts(g, E, 2 * I, H)[2:]
    w2 = _experts(g, E, H, I)[2:]
    a, ae, w, we, pre, desc = _dense(8, 64, 12544, 5)
    dws = bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, 8, 64, 12544)
    a2, ae2, w_2, we2, pre2, desc2 = _dense(200, 256, 4096, 6)
    dws2 = bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, 200, 256, 4096)
    ad, aed, a2d, ae2d = dev_u8(a), dev_u8(ae), dev_u8(a2), dev_u8(ae2)
    x = dev_bf16(synth.bf16_normal(g, (T, H), 1.0))
    many = 5000
    ids_many = torch.zeros((many, 2), dtype=torch.int32, device="cuda")
    sws = bs.alloc_workspace(bs.BS_OP_MOE_SORT, many, 2, E)
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    weights = torch.zeros((T, k), dtype=torch.float32, device="cuda")
    dout = dev_bf16(synth.bf16_normal(g, (T, H), 1.0))
    h = torch.zeros((T * k, 2 * I), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    dy, xs = torch.zeros_like(y), torch.zeros_like(y)

    def step():
        rows, pos, off = bs.moe_sort(ids, E)
        q, s = bs.quant_mxfp4(x)
        bs.bsgemm_w4a4_mxfp4_grouped(q, s, off, w1[1], w1[0], rows=rows, out=h)
        hq, hs = bs.silu_mul_quant_mxfp4(h, rows=off[E:])
        bs.bsgemm_w4a4_mxfp4_grouped(hq, hs, off, w2[1], w2[0], out=y)
        o = bs.moe_combine(y, pos, weights)
        _, dw = bs.moe_combine_backward(dout, y, pos, weights, dy=dy)
        bs.moe_gather(x, pos, out=xs)
        c = bs.bsgemm_w4a4_mxfp4(ad, aed, desc, pre, ws=dws)
        c2 = bs.bsgemm_w4a4_mxfp4(a2d, ae2d, desc2, pre2, ws=dws2)
        m = bs.moe_sort(ids_many, E, ws=sws)
        return [rows, pos, off, h, y, o, dw, dy, xs, c, c2, bs.dequant_mxfp4(q, s), *m]

    def new_inputs(i):
        gg = np.random.default_rng(100 + i)
        ids.copy_(torch.from_numpy(gg.integers(-1, E, (T, k)).astype(np.int32)))
        ids_many.copy_(torch.from_numpy(gg.integers(-1, E, (many, 2)).astype(np.int32)))
        weights.copy_(torch.from_numpy(gg.random((T, k), dtype=np.float32)))
        for b in (h, y, dy, xs):
            b.zero_()
    new_inputs(0)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            outs = step()
    torch.cuda.synchronize()
    for rep in range(4):
        new_inputs(rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        new_inputs(rep)
        want = step()
        torch.cuda.synchronize()
        for i, (u, v) in enumerate(zip(got, want)):
            assert torch.equal(u, v), f"replay {rep}, output {i}"


def test_runs_on_the_current_stream():
    """Work queued on a side stream is ordered there: the inputs are written by
    that stream just before the call."""
    M, N, K = 40, 64, 256
    a, ae, w, we, pre, desc = _dense(M, N, K, 8)
    src_a, src_e = dev_u8(a), dev_u8(ae)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ad, ed = torch.zeros_like(src_a), torch.zeros_like(src_e)
        for _ in range(20):
            ad.copy_(src_a)
        ed.copy_(src_e)
        c = bs.bsgemm_w4a4_mxfp4(ad, ed, desc, pre, ws=bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, M, N, K))
    side.synchronize()
    ce, asum = mxfp4.w4a4_gemm(a, ae, w, we)
    mxfp4.assert_w4a4_close(host_bits16(c), ce, asum, K)

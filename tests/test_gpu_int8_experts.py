"""The int8 and routing operators together, as a layer of experts runs them: norm
with int8 output, router, sort, the experts' products around the SiLU, combine; and
back from the output's gradient to the logits.  Eagerly, captured into a graph, on
two streams at once, and on buffers past 2^31 and 2^32 bytes."""
import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from oracle import codecs, int8, mxfp4, route
from tests.gpu_util import dev_bf16, host_bits16

pytestmark = pytest.mark.gpu


def _bf16(g, shape, std=1.0):
    return codecs.round_to_bf16(g.standard_normal(shape) * std)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """Weights of a layer (hidden H, experts' inner size I) and its calls."""

    def __init__(self, seed, E, H, I, k, groups=1, keep=1, top=1):
        g = np.random.default_rng(seed)
        self.E, self.H, self.I, self.k, self.groups, self.keep, self.top = E, H, I, k, groups, keep, top
        self.gamma = _bf16(g, (H,), 0.1)
        self.gate = _bf16(g, (E, H), H ** -0.5)
        self.bias = (g.standard_normal(E) * 0.02).astype(np.float32)
        self.w1 = [int8.quant_rows(codecs.decode_bf16(_bf16(g, (2 * I, H), 0.05))) for _ in range(E)]
        self.w2 = [int8.quant_rows(codecs.decode_bf16(_bf16(g, (H, I), 0.05))) for _ in range(E)]
        self.pre1, self.d1 = bs.prelayout_int8_experts(_dev(np.stack([w for w, _ in self.w1])))
        self.pre2, self.d2 = bs.prelayout_int8_experts(_dev(np.stack([w for w, _ in self.w2])))
        self.s1, self.s2 = _dev(np.stack([s for _, s in self.w1])), _dev(np.stack([s for _, s in self.w2]))
        self.dgamma, self.dgate, self.dbias = dev_bf16(self.gamma), dev_bf16(self.gate), _dev(self.bias)

    def logits(self, x):
        return (x.float() @ self.dgate.float().t()).contiguous()

    def run(self, y, res, logits, live=None, sort_ws=None):
        """Everything that the layer computes, in order."""
        q, s, r = bs.add_rms_quant_int8(y, res, self.dgamma)
        ids, weights = bs.moe_route(logits, self.k, bias=self.dbias, score=bs.BS_SCORE_SIGMOID, groups=self.groups,
                                    topk_groups=self.keep, group_top=self.top, scale=2.5, rows=live)
        rows, pos, off = bs.moe_sort(ids, self.E, ws=sort_ws)
        h = bs.bsgemm_w8a8_int8_grouped(q, s, off, self.d1, self.pre1, self.s1, rows=rows)
        hq, hs = bs.silu_mul_quant_int8(h, rows=off[self.E:])
        o = bs.bsgemm_w8a8_int8_grouped(hq, hs, off, self.d2, self.pre2, self.s2)
        out = bs.moe_combine(o, pos, weights)
        return dict(q=q, s=s, r=r, ids=ids, weights=weights, rows=rows, pos=pos, off=off, h=h, hq=hq, hs=hs, o=o, out=out)

    def backward(self, dout, st, logits):
        do, dw = bs.moe_combine_backward(dout, st["o"], st["pos"], st["weights"])
        return dw, bs.moe_route_backward(dw, logits, st["ids"], score=bs.BS_SCORE_SIGMOID, scale=2.5)


def _inputs(seed, T, H):
    g = np.random.default_rng(seed)
    return _bf16(g, (T, H)), _bf16(g, (T, H), 2.0)


@pytest.mark.parametrize("T,live,E,H,I,k,groups", [(1, None, 8, 128, 64, 2, 1), (7, 5, 16, 256, 96, 3, 4),
                                                    (300, 290, 12, 384, 80, 4, 3), (600, None, 64, 256, 128, 8, 8),
                                                    (5, 0, 8, 128, 64, 2, 2)])
def test_layer_against_the_oracle(T, live, E, H, I, k, groups):
    L = Layer(E + T, E, H, I, k, groups, max(1, groups // 2), 2 if groups > 1 else 1)
    y, res = _inputs(T, T, H)
    x = dev_bf16(y)
    logits = L.logits(x)
    dlive = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    st = L.run(x, dev_bf16(res), logits, dlive, bs.alloc_workspace(bs.BS_OP_MOE_SORT, T, k, E))
    torch.cuda.synchronize()
    # every stage from what the stage before it gave
    h, rb = int8.add_rms(y, res, L.gamma, 1e-6, 1.0)
    qo, so = int8.quant_rows(h)
    assert np.array_equal(st["q"].cpu().numpy(), qo) and np.array_equal(st["s"].cpu().numpy(), so)
    assert np.array_equal(host_bits16(st["r"]), rb)
    io, wo = route.route(logits.double().cpu().numpy(), k, L.bias, True, groups, L.keep, L.top, True, 2.5, live)
    assert np.array_equal(st["ids"].cpu().numpy(), io)
    w = st["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(w - wo) <= 8 * 2.0 ** -24 * wo).all()
    ro, po, oo = mxfp4.moe_sort(io, E)
    assert np.array_equal(st["rows"].cpu().numpy(), ro) and np.array_equal(st["pos"].cpu().numpy(), po)
    hb, ob, hq, hs = host_bits16(st["h"]), host_bits16(st["o"]), st["hq"].cpu().numpy(), st["hs"].cpu().numpy()
    used = oo[E]
    for e in range(E):
        r = slice(oo[e], oo[e + 1])
        if oo[e + 1] > oo[e]:
            assert np.array_equal(hb[r], int8.gemm(qo[ro[r]], so[ro[r]], *L.w1[e])), e
            assert np.array_equal(ob[r], int8.gemm(hq[r], hs[r], *L.w2[e])), e
    if used:
        q2, s2 = int8.quant_rows(int8.silu_mul(hb[:used]))
        assert np.array_equal(hq[:used], q2) and np.array_equal(hs[:used], s2)
    want, mag = mxfp4.moe_combine(codecs.decode_bf16(ob), po, w)
    got = codecs.decode_bf16(host_bits16(st["out"]))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2 * k * 2.0 ** -24 * mag + 2.0 ** -133).all()
    # back to the logits
    dout = dev_bf16(_bf16(np.random.default_rng(1), (T, H)))
    dw, dl = L.backward(dout, st, logits)
    torch.cuda.synchronize()
    wd, wm = route.route_backward(dw.double().cpu().numpy(), logits.double().cpu().numpy(), io, True, True, 2.5)
    off = np.abs(dl.double().cpu().numpy() - wd)
    assert (off <= 17 * 2.0 ** -24 * wm + 2.0 ** -133).all()
    if live is not None:
        assert not dl[live:].any() and not st["out"][live:].any()


def test_captured_and_replayed():
    """The layer and the dense product, captured once; replayed with new inputs in
    the captured buffers and eager work between."""
    T, E, H, I, k = 40, 16, 512, 128, 4
    L = Layer(3, E, H, I, k, 4, 2, 2)
    y, res = (dev_bf16(v) for v in _inputs(1, T, H))
    logits = L.logits(y)
    live = torch.tensor([T], dtype=torch.int32, device="cuda")
    g = np.random.default_rng(2)
    wq, wsc = int8.quant_rows(codecs.decode_bf16(_bf16(g, (96, 16384), 0.05)))
    pre, desc = bs.prelayout_int8(_dev(wq))
    dsc = _dev(wsc)
    ws = bs.alloc_workspace(bs.BS_OP_W8A8_INT8, 24, 96, 16384)
    assert ws is not None                                       # K is split through it
    a = dev_bf16(_bf16(g, (24, 16384)))
    dout = dev_bf16(_bf16(g, (T, H)))

    def call():
        st = L.run(y, res, logits, live)
        aq, asc = bs.quant_int8_per_token(a)
        c = bs.bsgemm_w8a8_int8(aq, asc, desc, pre, dsc, ws=ws)
        dw, dl = L.backward(dout, st, logits)
        return [st["out"], st["ids"], st["weights"], st["r"], c, dl, bs.dequant_int8(aq, asc)]
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for turn in range(5):
        y2, r2 = (dev_bf16(v) for v in _inputs(10 + turn, T, H))
        y.copy_(y2)
        res.copy_(r2)
        logits.copy_(L.logits(y2))
        live.fill_(T - 3 * turn)
        a.copy_(dev_bf16(_bf16(np.random.default_rng(turn), (24, 16384))))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = call()
        torch.cuda.synchronize()
        for i, (u, v) in enumerate(zip(got, want)):
            assert torch.equal(u, v), f"replay {turn}, output {i}"
        assert not ws[: 64 * 1024].any()


def test_two_streams_at_once():
    """Two layers on two streams, queued together several times, each with workspaces
    of its own: every result is that of a lone call."""
    T, E, H, I, k = 3000, 24, 256, 64, 2
    jobs = []
    for i in range(2):
        L = Layer(20 + i, E, H, I, k)
        y, res = (dev_bf16(v) for v in _inputs(30 + i, T, H))
        g = np.random.default_rng(40 + i)
        wq, wsc = int8.quant_rows(codecs.decode_bf16(_bf16(g, (64, 24576), 0.05)))
        aq, asc = int8.quant_rows(codecs.decode_bf16(_bf16(g, (20, 24576))))
        jobs.append((L, y, res, L.logits(y), bs.alloc_workspace(bs.BS_OP_MOE_SORT, T, k, E),
                     bs.prelayout_int8(_dev(wq)), _dev(wsc), _dev(aq), _dev(asc),
                     bs.alloc_workspace(bs.BS_OP_W8A8_INT8, 20, 64, 24576)))

    def run(j):
        L, y, res, logits, sws, (pre, desc), wsc, aq, asc, ws = j
        st = L.run(y, res, logits, sort_ws=sws)
        return [st["out"], st["ids"], st["weights"], bs.bsgemm_w8a8_int8(aq, asc, desc, pre, wsc, ws=ws)]
    want = [run(j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for j, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(run(j))
    torch.cuda.synchronize()
    for n, out in enumerate(got):
        for i, (u, v) in enumerate(zip(out, want[n % 2])):
            assert torch.equal(u, v), f"run {n}, output {i}"


def test_one_workspace_for_all_shapes():
    """One workspace, as large as the largest call needs, serves calls of other
    shapes and other operators in between."""
    shapes = [(8, 1000, 17408), (30, 200, 8192), (64, 1024, 16384), (3, 33, 131056), (16, 34816, 5120)]
    ws = torch.zeros(max(bs.workspace_bytes(bs.BS_OP_W8A8_INT8, *s) for s in shapes), dtype=torch.uint8, device="cuda")
    used = 0
    for turn in range(2):
        for M, N, K in shapes:
            g = np.random.default_rng(M + turn)
            a, w = (g.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (min(N, 128), K)))
            sa, sw = (np.exp(g.uniform(-9, -3, n)).astype(np.float32) for n in (M, min(N, 128)))
            reps = -(-N // len(w))
            pre, desc = bs.prelayout_int8(_dev(w).repeat(reps, 1)[:N].contiguous())
            c = bs.bsgemm_w8a8_int8(_dev(a), _dev(sa), desc, pre, _dev(sw).repeat(reps)[:N].contiguous(), ws=ws)
            want = np.tile(int8.gemm(a, sa, w, sw), (1, reps))[:, :N]
            assert np.array_equal(host_bits16(c), want), (M, N, K)
            used += bs.workspace_bytes(bs.BS_OP_W8A8_INT8, M, N, K) > 0
            assert not ws[: 64 * 1024].any()
    assert used >= 4


# ------------------------------------------------------------------ large buffers
@pytest.mark.parametrize("M", [3, 70])
def test_weight_and_output_past_2_31(M):
    """N * K = 4.4e9 bytes of weight: the same 16 rows 550000 times."""
    N, K = 16 * 550000, 512
    g = np.random.default_rng(M)
    a, w = g.integers(-128, 128, (M, K)).astype(np.int8), g.integers(-128, 128, (16, K)).astype(np.int8)
    sa, sw = (np.exp(g.uniform(-9, -3, n)).astype(np.float32) for n in (M, 16))
    pre, desc = bs.prelayout_int8(_dev(w).repeat(N // 16, 1))
    c = bs.bsgemm_w8a8_int8(_dev(a), _dev(sa), desc, pre, _dev(sw).repeat(N // 16),
                            ws=bs.alloc_workspace(bs.BS_OP_W8A8_INT8, M, N, K))
    torch.cuda.synchronize()
    assert np.array_equal(host_bits16(c[:, :16].contiguous()), int8.gemm(a, sa, w, sw))
    assert torch.equal(c.view(M, N // 16, 16), c[:, None, :16].expand(M, N // 16, 16))


def test_activation_and_output_past_2_32():
    """300000 rows 16000 bytes apart, and as many output rows of 8000."""
    M, N, K, lda, ldc = 300000, 64, 256, 16000, 8000
    g = np.random.default_rng(1)
    a, w = g.integers(-128, 128, (400, K)).astype(np.int8), g.integers(-128, 128, (N, K)).astype(np.int8)
    sa, sw = (np.exp(g.uniform(-9, -3, n)).astype(np.float32) for n in (400, N))
    buf = torch.zeros(((M - 1) * lda + K,), dtype=torch.int8, device="cuda")
    wide = buf.as_strided((M, K), (lda, 1))
    wide.copy_(_dev(a).repeat(M // 400, 1))
    out = torch.empty((M, ldc), dtype=torch.bfloat16, device="cuda")[:, :N]
    pre, desc = bs.prelayout_int8(_dev(w))
    bs.bsgemm_w8a8_int8(wide, _dev(sa).repeat(M // 400), desc, pre, _dev(sw), out=out)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits16(out[:400].contiguous()), int8.gemm(a, sa, w, sw))
    assert torch.equal(out.unflatten(0, (M // 400, 400)), out[None, :400].expand(M // 400, 400, N))


@pytest.mark.parametrize("per", [2, 30, 100])
def test_experts_past_2_32_bytes(per):
    """Four experts 1.5e9 bytes apart; each row regime of the grouped product."""
    E, N, K, stride = 4, 80, 384, 1_500_000_000 // 256 * 256
    g = np.random.default_rng(per)
    w, sw = g.integers(-128, 128, (E, N, K)).astype(np.int8), np.exp(g.uniform(-9, -3, (E, N))).astype(np.float32)
    pre, desc = bs.prelayout_int8_experts(_dev(w))
    nb = pre.shape[1]
    buf = torch.zeros(((E - 1) * stride + nb,), dtype=torch.uint8, device="cuda")
    wide = buf.as_strided((E, nb), (stride, 1))
    wide.copy_(pre)
    S = E * per
    a, sa = g.integers(-128, 128, (S, K)).astype(np.int8), np.exp(g.uniform(-9, -3, S)).astype(np.float32)
    off = torch.arange(0, S + 1, per, dtype=torch.int32, device="cuda")
    c = host_bits16(bs.bsgemm_w8a8_int8_grouped(_dev(a), _dev(sa), off, desc, wide, _dev(sw)))
    for e in range(E):
        r = slice(e * per, (e + 1) * per)
        assert np.array_equal(c[r], int8.gemm(a[r], sa[r], w[e], sw[e])), e


def test_gathered_rows_past_2_31_bytes():
    """Rows of the activation up to byte 4.2e9, gathered through the order."""
    Ma, K, lda, N = 260, 128, 16_515_056, 48
    g = np.random.default_rng(5)
    a, sa = g.integers(-128, 128, (Ma, K)).astype(np.int8), np.exp(g.uniform(-9, -3, Ma)).astype(np.float32)
    buf = torch.zeros(((Ma - 1) * lda + K,), dtype=torch.int8, device="cuda")
    wide = buf.as_strided((Ma, K), (lda, 1))
    wide.copy_(_dev(a))
    for E, S in ((40, 60), (1, 200), (2, 500)):
        w, sw = g.integers(-128, 128, (E, N, K)).astype(np.int8), np.exp(g.uniform(-9, -3, (E, N))).astype(np.float32)
        pre, desc = bs.prelayout_int8_experts(_dev(w))
        rows = g.integers(0, Ma, S).astype(np.int32)
        rows[-1] = Ma - 1
        off = np.sort(np.concatenate([[0], g.integers(0, S + 1, E - 1), [S]])).astype(np.int32)
        c = host_bits16(bs.bsgemm_w8a8_int8_grouped(wide, _dev(sa), _dev(off), desc, pre, _dev(sw), rows=_dev(rows)))
        for e in range(E):
            r = rows[off[e]:off[e + 1]]
            assert np.array_equal(c[off[e]:off[e + 1]], int8.gemm(a[r], sa[r], w[e], sw[e])), (E, e)


def test_quantisers_past_2_31_values():
    """270000 rows of 8192 (2.2e9 values): a pattern of 240 rows repeated."""
    P, R, K = 240, 1125, 8192
    g = np.random.default_rng(9)
    bits = _bf16(g, (P, 2 * K))
    gu = dev_bf16(bits).repeat(R, 1)
    q, s = bs.silu_mul_quant_int8(gu)
    qo, so = int8.quant_rows(int8.silu_mul(bits))

    def same():
        assert np.array_equal(q[:P].cpu().numpy(), qo) and np.array_equal(s[:P].cpu().numpy(), so)
        assert torch.equal(q.view(R, P, K), q[None, :P].expand(R, P, K)) and torch.equal(s.view(R, P), s[None, :P].expand(R, P))
    same()
    bs.quant_int8_per_token(gu[:, :K], q, s)                    # strided rows
    qo, so = int8.quant_rows(codecs.decode_bf16(bits[:, :K]))
    same()
    # as rows of K: row i of the pattern's 2 P; R is odd, so y's row i meets row i + P of the pattern
    x, rows = gu.view(2 * R * P, K), bits.reshape(2 * P, K)
    gamma = _bf16(g, (K,), .1)
    q, s, r = bs.add_rms_quant_int8(x[: R * P], x[R * P:], dev_bf16(gamma))
    h, rb = int8.add_rms(rows[:P], rows[P:], gamma, 1e-6, 1.0)
    qo, so = int8.quant_rows(h)
    same()
    assert np.array_equal(host_bits16(r[:P]), rb) and torch.equal(r.view(R, P, K), r[None, :P].expand(R, P, K))
    assert torch.equal(bs.dequant_int8(q, s)[-P:], bs.dequant_int8(q[-P:].contiguous(), s[-P:].contiguous()))


def test_logits_past_2_32_bytes():
    """1100000 tokens of 1024 fp32 logits: a pattern of 1000 tokens repeated."""
    P, R, E, k = 1000, 1100, 1024, 3
    pat = torch.randn((P, E), generator=torch.Generator().manual_seed(1)).cuda()
    x = pat.repeat(R, 1)
    ids, w = bs.moe_route(x, k)
    io, wo = route.route(pat[:50].double().cpu().numpy(), k)
    assert np.array_equal(ids[:50].cpu().numpy(), io)
    assert torch.equal(ids.view(R, P, k), ids[None, :P].expand(R, P, k)) and torch.equal(w.view(R, P, k), w[None, :P].expand(R, P, k))
    dw = torch.randn((P, k), generator=torch.Generator().manual_seed(2)).cuda().repeat(R, 1)
    d = bs.moe_route_backward(dw, x, ids, renorm=False)
    want, mag = route.route_backward(dw[:20].double().cpu().numpy(), pat[:20].double().cpu().numpy(), io[:20], False, False, 1.0)
    assert (np.abs(d[:20].double().cpu().numpy() - want) <= 17 * 2.0 ** -24 * mag + 2.0 ** -133).all()
    assert torch.equal(d.view(R, P, E), d[None, :P].expand(R, P, E))

"""int8 producers against the oracle: codes and scales bit for bit (every step of
the kernels but one rounding of h is exact, and h is the real value rounded once),
the residual and the values read back too."""
import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from oracle import codecs, int8
from tests.gpu_util import dev_bf16, host_bits16

pytestmark = pytest.mark.gpu


def _bf16(seed, shape, std=1.0, outliers=0.002):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * std
    x *= np.where(g.random(shape) < outliers, 16.0, 1.0)
    return codecs.round_to_bf16(x)


def _same(q, s, h, what=""):
    qo, so = int8.quant_rows(h)
    torch.cuda.synchronize()
    assert np.array_equal(s.cpu().numpy(), so, equal_nan=True), f"{what}: scales"
    got = q.cpu().numpy()
    bad = np.argwhere(got != qo)
    assert not len(bad), f"{what}: {len(bad)} codes differ, first {bad[:3].tolist()}"


SIZES = [(1, 8), (1, 16), (3, 24), (7, 520), (5, 2040), (4, 2048), (9, 2056), (300, 5120), (2, 17408), (3, 32760),
         (2, 32768), (2500, 128), (2100, 5120), (1, 5120)]


@pytest.mark.parametrize("M,K", SIZES)
def test_quant_per_token(M, K):
    x = _bf16(M + K, (M, K), 3.0)
    q, s = bs.quant_int8_per_token(dev_bf16(x))
    _same(q, s, codecs.decode_bf16(x), f"{M}x{K}")


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("offset,residual", [(1.0, True), (0.0, True), (0.0, False), (1.0, False)])
def test_add_rms(M, K, offset, residual):
    y, r, g = _bf16(M, (M, K)), _bf16(K, (M, K), 2.0), _bf16(1, (K,), .2, 0)
    if offset == 0.0:
        g = _bf16(2, (K,), 1.0, 0)
    q, s, ro = bs.add_rms_quant_int8(dev_bf16(y), dev_bf16(r) if residual else None, dev_bf16(g), 1e-6, offset)
    h, rb = int8.add_rms(y, r if residual else None, g, 1e-6, offset)
    _same(q, s, h, f"{M}x{K}")
    if residual:
        assert np.array_equal(host_bits16(ro), rb)
    else:
        assert ro is None


@pytest.mark.parametrize("M,N", SIZES)
def test_silu_mul(M, N):
    gu = _bf16(M * 3 + N, (M, 2 * N), 1.5)
    q, s = bs.silu_mul_quant_int8(dev_bf16(gu))
    _same(q, s, int8.silu_mul(gu), f"{M}x{N}")


def test_every_bf16_value():
    """Rows whose maximum is every finite bf16 magnitude, with quotients on and next
    to the middle between two codes."""
    top = np.arange(0, 0x7F80, 3, dtype=np.uint16)
    v = codecs.decode_bf16(top)
    g = np.random.default_rng(0)
    x = v[:, None] * (g.integers(-254, 255, (len(top), 32)) / 254.0)
    x[:, 0] = v
    x = codecs.round_to_bf16(x)
    x[:, 0] = top
    q, s = bs.quant_int8_per_token(dev_bf16(x))
    _same(q, s, codecs.decode_bf16(x))


def test_ties():
    """A scale of one (and of a power of two): halves round to the even code."""
    g = np.random.default_rng(1)
    for e in (-100, 0, 60):
        x = g.integers(-253, 254, (64, 256)) / 2.0
        x[:, 7] = 127.0
        b = codecs.round_to_bf16(x * 2.0 ** e)
        q, s = bs.quant_int8_per_token(dev_bf16(b))
        _same(q, s, codecs.decode_bf16(b))


def test_silu_extremes():
    """Gates over the whole range of bf16 (zeros, subnormals, the largest values),
    products that leave fp32's range, rows near the floor of the scale."""
    g = np.random.default_rng(2)
    gate = np.concatenate([np.arange(0, 0x7F80, 7), np.arange(0x8000, 0xFF80, 7)]).astype(np.uint16)
    rows = []
    for up in (0x3F80, 0xBF81, 0x0001, 0x0080, 0x0000, 0x7F00, 0x2000, 0x5F80):
        rows.append(np.stack([gate, np.full_like(gate, up)]))
    n = len(gate) // 8 * 8
    gu = np.stack([np.concatenate([r[0][:n], r[1][:n]]) for r in rows])
    q, s = bs.silu_mul_quant_int8(dev_bf16(gu))
    _same(q, s, int8.silu_mul(gu))
    # the same gates a few to a row, so that small rows have scales of their own
    order = g.permutation(n)
    for up in (0x3F80, 0x0001, 0x2000):
        small = np.sort(gate[:n])[: n // 8 * 8].reshape(-1, 8)
        gu = np.concatenate([small, np.full_like(small, up)], axis=1)
        q, s = bs.silu_mul_quant_int8(dev_bf16(gu))
        _same(q, s, int8.silu_mul(gu), hex(up))
    mixed = np.concatenate([gate[order].reshape(-1, 8), gate[g.permutation(n)].reshape(-1, 8)], axis=1)
    q, s = bs.silu_mul_quant_int8(dev_bf16(mixed))
    _same(q, s, int8.silu_mul(mixed), "mixed")


def test_not_finite():
    """Rows with an infinity or a NaN: a NaN scale, zero codes; their neighbours as ever."""
    x = _bf16(5, (6, 256))
    x[1, 3], x[2, 100], x[4, 255] = 0x7F80, 0x7FC1, 0xFF80
    q, s = bs.quant_int8_per_token(dev_bf16(x))
    _same(q, s, codecs.decode_bf16(x))
    assert np.isnan(s.cpu().numpy()[[1, 2, 4]]).all()
    r, g = _bf16(6, (6, 256)), _bf16(7, (256,), .1)
    q, s, _ = bs.add_rms_quant_int8(dev_bf16(x), dev_bf16(r), dev_bf16(g))
    h, _ = int8.add_rms(x, r, g, 1e-6, 1.0)
    _same(q, s, h)
    gu = _bf16(8, (5, 512))
    gu[0, 9], gu[1, 300], gu[2, 5], gu[3, 511] = 0x7F80, 0x7FC0, 0xFF80, 0xFF80
    gu[3, 255] = 0                              # 0 * inf
    q, s = bs.silu_mul_quant_int8(dev_bf16(gu))
    _same(q, s, int8.silu_mul(gu))
    d = bs.dequant_int8(q, s)
    assert torch.isnan(d[:4].float()).all() and torch.isfinite(d[4].float()).all()


def test_zero_rows_and_small_norms():
    y = np.zeros((3, 64), np.uint16)
    y[1] = codecs.round_to_bf16(np.full(64, 1e-20))
    y[2, 5] = codecs.round_to_bf16(np.array([1e-30]))[0]
    g = _bf16(1, (64,), .1)
    for eps in (0.0, 1e-6):
        h, _ = int8.add_rms(y, y, g, eps, 1.0)
        q, s, _ = bs.add_rms_quant_int8(dev_bf16(y), dev_bf16(y), dev_bf16(g), eps)
        _same(q, s, h, f"eps {eps}")


def test_residual_in_place_and_outputs():
    y, r, g = _bf16(1, (33, 1024)), _bf16(2, (33, 1024)), _bf16(3, (1024,), .1)
    h, rb = int8.add_rms(y, r, g, 1e-5, 1.0)
    res = dev_bf16(r)
    q, s = torch.empty((33, 1024), dtype=torch.int8, device="cuda"), torch.empty(33, device="cuda")
    out = bs.add_rms_quant_int8(dev_bf16(y), res, dev_bf16(g), 1e-5, q=q, scale=s, residual_out=res)
    assert out[0] is q and out[1] is s and out[2] is res
    _same(q, s, h)
    assert np.array_equal(host_bits16(res), rb)


def test_strides_and_alignment():
    base = dev_bf16(_bf16(9, (40, 1100)))
    for view in (base[:, :1024], base[::2, 8:520], base[:, 4:1028], base[:8, ::2][:, :512], base.t()[:64, :40],
                 base[3:4, 16:800]):
        q, s = bs.quant_int8_per_token(view)
        _same(q, s, view.float().cpu().numpy().astype(np.float64))
    gu = base[:, 1:1025]
    q, s = bs.silu_mul_quant_int8(gu)
    _same(q, s, int8.silu_mul(host_bits16(gu.contiguous())))
    q, s, ro = bs.add_rms_quant_int8(base[:, 1:513], base[:, 3:515], base[0, 5:517])
    h, rb = int8.add_rms(host_bits16(base[:, 1:513].contiguous()), host_bits16(base[:, 3:515].contiguous()),
                         host_bits16(base[0, 5:517].contiguous()), 1e-6, 1.0)
    _same(q, s, h)
    assert np.array_equal(host_bits16(ro), rb)


@pytest.mark.parametrize("live", [0, 1, 5, 8, 11, -3])
def test_silu_rows_on_the_device(live):
    gu = _bf16(4, (8, 512))
    q = torch.full((8, 256), 99, dtype=torch.int8, device="cuda")
    s = torch.full((8,), 7.0, device="cuda")
    bs.silu_mul_quant_int8(dev_bf16(gu), q=q, scale=s, rows=torch.tensor([live], dtype=torch.int32, device="cuda"))
    n = min(max(live, 0), 8)
    if n:
        _same(q[:n], s[:n], int8.silu_mul(gu[:n]))
    assert bool((q[n:] == 99).all()) and bool((s[n:] == 7.0).all())


@pytest.mark.parametrize("M,K", [(1, 8), (7, 520), (300, 5120), (4099, 136)])
def test_dequant(M, K):
    g = np.random.default_rng(M)
    q = g.integers(-128, 128, (M, K)).astype(np.int8)
    s = (np.exp(g.uniform(-40, 40, M))).astype(np.float32)
    out = bs.dequant_int8(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    assert np.array_equal(host_bits16(out), int8.dequant(q, s))


def test_dequant_rounds_once():
    """Every code times many scales: products next to the middle between two bf16
    values round by the exact product; beyond the range to infinities."""
    g = np.random.default_rng(3)
    q = np.tile(np.arange(-128, 128, dtype=np.int8), (4096, 1))
    s = (g.integers(1 << 23, 1 << 24, 4096) * 2.0 ** g.integers(-149, 100, 4096)).astype(np.float32)
    s[:3] = [3.3e38, np.float32(2.0 ** -149), np.float32("inf")]
    q[2] = 5
    out = bs.dequant_int8(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    assert np.array_equal(host_bits16(out), int8.dequant(q, s))


def test_empty():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    q, s = bs.quant_int8_per_token(e)
    assert q.shape == (0, 64) and s.shape == (0,)
    assert bs.dequant_int8(q, s).shape == (0, 64)
    assert bs.silu_mul_quant_int8(e)[0].shape == (0, 32)
    assert bs.add_rms_quant_int8(e, e, e.new_zeros(64))[2].shape == (0, 64)

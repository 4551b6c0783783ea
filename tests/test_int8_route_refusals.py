"""Every argument check of the int8 and routing calls of the binding, each by its own
message.  CPU only: the check of the device is switched off and the library replaced by
one that no call may reach, so that neither a tensor on the host nor the C side's checks
stand in for the one that a case is about."""
import pytest
import torch

import block_scaled_precision_04_amd as bs
from block_scaled_precision_04_amd import _binding
from block_scaled_precision_04_amd._binding import WDesc, BS_WDESC_MAGIC, BS_LAYOUT_INT8

N, K, E = 256, 512, 2
BYTES = N * K


def _desc():
    return WDesc(BS_WDESC_MAGIC, BS_LAYOUT_INT8, N, K, BYTES, 0, 0, BYTES)


def _t(dtype):
    return lambda *shape: torch.zeros(shape, dtype=dtype)


_i8, _u8, _f32, _bf, _i32, _i64 = (_t(d) for d in (torch.int8, torch.uint8, torch.float32, torch.bfloat16, torch.int32, torch.int64))


def _dense(**kw):
    a = dict(a=_i8(4, K), a_scale=_f32(4), desc=_desc(), w_pre=_u8(BYTES), w_scale=_f32(N))
    a.update(kw)
    return lambda: bs.bsgemm_w8a8_int8(**a)


def _grouped(**kw):
    a = dict(a=_i8(4, K), a_scale=_f32(4), offsets=_i32(E + 1), desc=_desc(), w_pre=_u8(E, BYTES), w_scale=_f32(E, N))
    a.update(kw)
    return lambda: bs.bsgemm_w8a8_int8_grouped(**a)


def _quant(**kw):
    a = dict(x=_bf(4, 64))
    a.update(kw)
    return lambda: bs.quant_int8_per_token(**a)


def _norm(**kw):
    a = dict(y=_bf(4, 64), residual=_bf(4, 64), gamma=_bf(64))
    a.update(kw)
    return lambda: bs.add_rms_quant_int8(**a)


def _silu(**kw):
    a = dict(gu=_bf(4, 128))
    a.update(kw)
    return lambda: bs.silu_mul_quant_int8(**a)


def _dequant(**kw):
    a = dict(q=_i8(4, 64), scale=_f32(4))
    a.update(kw)
    return lambda: bs.dequant_int8(**a)


def _route(**kw):
    a = dict(logits=_f32(4, 8), k=2)
    a.update(kw)
    return lambda: bs.moe_route(**a)


def _back(**kw):
    a = dict(dweights=_f32(4, 2), logits=_f32(4, 8), ids=_i32(4, 2))
    a.update(kw)
    return lambda: bs.moe_route_backward(**a)


HOST = r"tensors must be on a GPU, got \['cpu'\]"
REFUSED = {
    # dense product
    "a list": (_dense(a=[1]), "a must be a 2-D tensor"),
    "a 1-D": (_dense(a=_i8(K)), "a must be a 2-D tensor"),
    "a uint8": (_dense(a=_u8(4, K)), "a has dtype torch.uint8"),
    "a K": (_dense(a=_i8(4, K + 16)), "a has K = 528, the weight descriptor K = 512"),
    "a columns": (_dense(a=_i8(4, 2 * K)[:, ::2]), "a must have unit stride"),
    "a rows overlap": (_dense(a=_i8(K + 64).as_strided((4, K), (16, 1))), "a rows overlap"),
    "a_scale none": (_dense(a_scale=None), "a_scale is required"),
    "a_scale shape": (_dense(a_scale=_f32(5)), r"a_scale has shape \(5,\), expected \(4,\)"),
    "a_scale column": (_dense(a_scale=_f32(4, 1)), "a_scale has shape"),
    "a_scale bf16": (_dense(a_scale=_bf(4)), "a_scale has dtype"),
    "a_scale stride": (_dense(a_scale=_f32(8)[::2]), "a_scale must be contiguous"),
    "w_pre none": (_dense(w_pre=None), "w_pre must be a torch.Tensor"),
    "w_pre short": (_dense(w_pre=_u8(BYTES - 1)), "w_pre holds 131071 bytes, the layout needs 131072"),
    "w_pre int8": (_dense(w_pre=_i8(BYTES)), "w_pre has dtype torch.int8"),
    "w_pre 2-D": (_dense(w_pre=_u8(N, K)), "w_pre has shape"),
    "w_pre stride": (_dense(w_pre=_u8(2 * BYTES)[::2]), "w_pre must be contiguous"),
    "w_scale shape": (_dense(w_scale=_f32(N - 1)), "w_scale has shape"),
    "w_scale fp64": (_dense(w_scale=_t(torch.float64)(N)), "w_scale has dtype"),
    "w_scale stride": (_dense(w_scale=_f32(2 * N)[::2]), "w_scale must be contiguous"),
    "out fp32": (_dense(out=_f32(4, N)), "out has dtype"),
    "out shape": (_dense(out=_bf(4, N + 1)), "out has shape"),
    "out columns": (_dense(out=_bf(4, 2 * N)[:, ::2]), "out must have unit stride"),
    "out rows overlap": (_dense(out=_bf(N + 64).as_strided((4, N), (16, 1))), "out rows overlap"),
    "ws stride": (_dense(ws=_u8(64, 64)[:, ::2]), "ws must be a contiguous tensor"),
    "ws list": (_dense(ws=[0]), "ws must be a contiguous tensor"),
    # by expert
    "grouped a uint8": (_grouped(a=_u8(4, K)), "a has dtype torch.uint8"),
    "grouped a K": (_grouped(a=_i8(4, K - 16)), "a has K = 496"),
    "grouped a_scale": (_grouped(a_scale=_f32(3)), "a_scale has shape"),
    "grouped w_pre 1-D": (_grouped(w_pre=_u8(E * BYTES)), "w_pre must be a 2-D tensor"),
    "grouped w_pre int8": (_grouped(w_pre=_i8(E, BYTES)), "w_pre has dtype"),
    "grouped w_pre short": (_grouped(w_pre=_u8(E, BYTES - 256)), "w_pre holds 130816 bytes an expert"),
    "grouped w_pre columns": (_grouped(w_pre=_u8(E, 2 * BYTES)[:, ::2]), "w_pre must have unit stride"),
    "grouped w_pre overlaps": (_grouped(w_pre=_u8(BYTES + 256).as_strided((E, BYTES), (256, 1))), "w_pre rows overlap"),
    "grouped w_scale flat": (_grouped(w_scale=_f32(E * N)), "w_scale has shape"),
    "grouped w_scale bf16": (_grouped(w_scale=_bf(E, N)), "w_scale has dtype"),
    "grouped w_scale stride": (_grouped(w_scale=_f32(E, 2 * N)[:, :N]), "w_scale must be contiguous"),
    "offsets short": (_grouped(offsets=_i32(E)), "offsets has shape"),
    "offsets int64": (_grouped(offsets=_i64(E + 1)), "offsets has dtype"),
    "offsets stride": (_grouped(offsets=_i32(2 * E + 2)[::2]), "offsets must be contiguous"),
    "grouped rows list": (_grouped(rows=[0, 1]), "rows must be a torch.Tensor"),
    "grouped rows int64": (_grouped(rows=_i64(4)), "rows has dtype"),
    "grouped rows 2-D": (_grouped(rows=_i32(2, 2)), "rows has shape"),
    "grouped rows stride": (_grouped(rows=_i32(8)[::2]), "rows must be contiguous"),
    "grouped out shape": (_grouped(out=_bf(5, N)), "out has shape"),
    "grouped out rows": (_grouped(rows=_i32(6), out=_bf(4, N)), r"out has shape \(4, 256\), expected \(6, 256\)"),
    "grouped out fp32": (_grouped(out=_f32(4, N)), "out has dtype"),
    # layouts
    "prelayout 1-D": (lambda: bs.prelayout_int8(_i8(64)), "w must be a 2-D tensor"),
    "prelayout uint8": (lambda: bs.prelayout_int8(_u8(16, 64)), "prelayout_int8: w has dtype torch.uint8"),
    "experts 2-D": (lambda: bs.prelayout_int8_experts(_i8(16, 64)), "w must be a 3-D tensor"),
    "experts bf16": (lambda: bs.prelayout_int8_experts(_bf(2, 16, 64)), "prelayout_int8_experts: w has dtype"),
    "no experts": (lambda: bs.prelayout_int8_experts(_i8(0, 16, 64)), "at least one expert"),
    "unprelayout list": (lambda: bs.unprelayout_int8(_desc(), [0]), "pre must be a torch.Tensor"),
    "unprelayout int8": (lambda: bs.unprelayout_int8(_desc(), _i8(BYTES)), "pre has dtype"),
    "unprelayout stride": (lambda: bs.unprelayout_int8(_desc(), _u8(2 * BYTES)[::2]), "pre must be contiguous"),
    "unprelayout short": (lambda: bs.unprelayout_int8(_desc(), _u8(BYTES - 1)), "pre holds 131071 bytes, the layout needs 131072"),
    # producers
    "quant 1-D": (_quant(x=_bf(64)), "x must be a 2-D tensor"),
    "quant list": (_quant(x=[1.0]), "x must be a 2-D tensor"),
    "quant fp32": (_quant(x=_f32(4, 64)), "x has dtype"),
    "quant q bf16": (_quant(q=_bf(4, 64)), "q has dtype"),
    "quant q shape": (_quant(q=_i8(4, 63)), "q has shape"),
    "quant q stride": (_quant(q=_i8(4, 80)[:, :64]), "q must be contiguous"),
    "quant scale fp64": (_quant(scale=_t(torch.float64)(4)), "scale has dtype"),
    "quant scale shape": (_quant(scale=_f32(3)), "scale has shape"),
    "quant scale stride": (_quant(scale=_f32(8)[::2]), "scale must be contiguous"),
    "norm y fp32": (_norm(y=_f32(4, 64)), "y has dtype"),
    "norm y 1-D": (_norm(y=_bf(64)), "y must be a 2-D tensor"),
    "norm gamma shape": (_norm(gamma=_bf(65)), "gamma has shape"),
    "norm gamma fp32": (_norm(gamma=_f32(64)), "gamma has dtype"),
    "norm gamma none": (_norm(gamma=None), "gamma is required"),
    "norm residual shape": (_norm(residual=_bf(3, 64)), "residual has shape"),
    "norm residual fp32": (_norm(residual=_f32(4, 64)), "residual has dtype"),
    "norm residual_out shape": (_norm(residual_out=_bf(4, 65)), "residual_out has shape"),
    "norm residual_out fp32": (_norm(residual_out=_f32(4, 64)), "residual_out has dtype"),
    "norm residual_out stride": (_norm(residual_out=_bf(4, 80)[:, :64]), "residual_out must be contiguous"),
    "norm q": (_norm(q=_u8(4, 64)), "q has dtype"),
    "norm scale": (_norm(scale=_f32(4, 1)), "scale has shape"),
    "silu fp32": (_silu(gu=_f32(4, 128)), "gu has dtype"),
    "silu odd": (_silu(gu=_bf(4, 127)), r"gu must be a 2-D tensor \[M, 2N\]"),
    "silu q": (_silu(q=_i8(4, 128)), "q has shape"),
    "silu scale": (_silu(scale=_bf(4)), "scale has dtype"),
    "silu rows": (_silu(rows=_i32(2)), "rows has shape"),
    "silu rows int64": (_silu(rows=_i64(1)), "rows has dtype"),
    "dequant 1-D": (_dequant(q=_i8(64)), "q must be a 2-D tensor"),
    "dequant uint8": (_dequant(q=_u8(4, 64)), "q has dtype"),
    "dequant scale shape": (_dequant(scale=_f32(5)), "scale has shape"),
    "dequant scale bf16": (_dequant(scale=_bf(4)), "scale has dtype"),
    "dequant scale stride": (_dequant(scale=_f32(8)[::2]), "scale must be contiguous"),
    "dequant out fp32": (_dequant(out=_f32(4, 64)), "out has dtype"),
    "dequant out shape": (_dequant(out=_bf(4, 72)), "out has shape"),
    "dequant out stride": (_dequant(out=_bf(4, 80)[:, :64]), "out must be contiguous"),
    # routing
    "route 1-D": (_route(logits=_f32(8)), "logits must be a 2-D tensor"),
    "route fp16": (_route(logits=_t(torch.float16)(4, 8)), "logits has dtype torch.float16"),
    "route columns": (_route(logits=_f32(4, 16)[:, ::2]), "logits must have unit stride"),
    "route rows overlap": (_route(logits=_f32(20).as_strided((4, 8), (4, 1))), "logits rows overlap"),
    "route k": (_route(k=0), "k = 0 must be a positive int"),
    "route k float": (_route(k=2.0), "k = 2.0 must be a positive int"),
    "route groups": (_route(groups=0), "groups = 0 must be a positive int"),
    "route topk_groups": (_route(topk_groups=-1), "topk_groups = -1 must be a positive int"),
    "route group_top": (_route(group_top=0), "group_top = 0 must be a positive int"),
    "route bias bf16": (_route(bias=_bf(8)), "bias has dtype"),
    "route bias shape": (_route(bias=_f32(4, 8)), "bias has shape"),
    "route bias stride": (_route(bias=_f32(16)[::2]), "bias must be contiguous"),
    "route rows": (_route(rows=_i32(4)), "rows has shape"),
    "route rows int64": (_route(rows=_i64(1)), "rows has dtype"),
    "route ids shape": (_route(ids=_i32(4, 3)), "ids has shape"),
    "route ids int64": (_route(ids=_i64(4, 2)), "ids has dtype"),
    "route ids stride": (_route(ids=_i32(4, 4)[:, :2]), "ids must be contiguous"),
    "route weights shape": (_route(weights=_f32(3, 2)), "weights has shape"),
    "route weights bf16": (_route(weights=_bf(4, 2)), "weights has dtype"),
    "route weights stride": (_route(weights=_f32(4, 4)[:, :2]), "weights must be contiguous"),
    "backward logits": (_back(logits=_i32(4, 8)), "logits has dtype"),
    "backward ids 1-D": (_back(ids=_i32(8)), "ids must be a 2-D tensor"),
    "backward ids tokens": (_back(ids=_i32(3, 2), dweights=_f32(3, 2)), r"ids has shape \(3, 2\), expected \(4, 2\)"),
    "backward ids fp32": (_back(ids=_f32(4, 2)), "ids has dtype"),
    "backward ids stride": (_back(ids=_i32(4, 4)[:, :2]), "ids must be contiguous"),
    "backward dweights shape": (_back(dweights=_f32(4, 3)), "dweights has shape"),
    "backward dweights bf16": (_back(dweights=_bf(4, 2)), "dweights has dtype"),
    "backward dweights stride": (_back(dweights=_f32(4, 4)[:, :2]), "dweights must be contiguous"),
    "backward dlogits 1-D": (_back(dlogits=_f32(32)), "dlogits must be a 2-D tensor"),
    "backward dlogits type": (_back(dlogits=_bf(4, 8)), "dlogits has dtype torch.bfloat16, the logits torch.float32"),
    "backward dlogits shape": (_back(dlogits=_f32(4, 9)), "dlogits has shape"),
    "backward dlogits rows": (_back(dlogits=_f32(20).as_strided((4, 8), (4, 1))), "dlogits rows overlap"),
}


class _NoLibrary:
    def bs_prelayout_int8_bytes(self, n, k):
        return 2048

    def __getattr__(self, name):
        raise AssertionError(f"nothing refused the call before {name}")


@pytest.mark.parametrize("case", REFUSED)
def test_refused_by_its_own_check(monkeypatch, case):
    call, message = REFUSED[case]
    monkeypatch.setattr(_binding, "_on_current", lambda fn, *ts: 0)
    monkeypatch.setattr(_binding, "_stream_of", lambda dev: 0)
    monkeypatch.setattr(_binding, "lib", _NoLibrary)
    with pytest.raises(ValueError, match=message):
        call()


@pytest.mark.parametrize("call", [
    _dense(), _grouped(), lambda: bs.prelayout_int8(_i8(16, 64)), lambda: bs.unprelayout_int8(_desc(), _u8(BYTES)), _quant(),
    _norm(), _norm(residual=None), _silu(), _dequant(), _route(), _back()],
    ids=["dense", "grouped", "prelayout", "unprelayout", "quant", "norm", "norm alone", "silu", "dequant", "route", "backward"])
def test_host_tensors_are_refused(monkeypatch, call):
    monkeypatch.setattr(_binding, "lib", _NoLibrary)
    with pytest.raises(ValueError, match=HOST):
        call()


@pytest.mark.parametrize("call", [_dense(), _grouped(), _quant(), _norm(), _silu(), _dequant(), _route(), _back(),
                                  lambda: bs.prelayout_int8(_i8(16, 64)), lambda: bs.unprelayout_int8(_desc(), _u8(BYTES))])
def test_the_same_calls_without_a_mistake_reach_the_library(monkeypatch, call):
    """What the cases above change is all that is wrong with them."""
    monkeypatch.setattr(_binding, "_on_current", lambda fn, *ts: 0)
    monkeypatch.setattr(_binding, "_stream_of", lambda dev: 0)
    monkeypatch.setattr(_binding, "lib", _NoLibrary)
    with pytest.raises(AssertionError, match="nothing refused the call"):
        call()

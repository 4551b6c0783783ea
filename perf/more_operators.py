"""Cases that time the int8 (W8A8) operators and the routing to experts.

Every case runs one operator on inputs made from a seed.  With ``own`` false
the operator is computed in its plain form (elementary torch operations); with
``own`` true through the library's entry points, as a program would call them.

Kinds of case:
  route           logits [T, E] -> the k experts of each token and their weights
  route_backward  the gradient of the weights back to the logits
  norm            residual add, RMS norm, int8 codes with a scale per token; the
                  codes read back as bf16, the values they stand for
  silu            SiLU(gate) * up from a gate/up projection's output [M, 2K],
                  the same codes, read back
  gemm            C = A . W^T, int8 with a scale per token and output channel
  grouped         the experts' products on the sorted rows (rows read through
                  the order, weights of all experts in one buffer)

K is the inner size, N the output columns, T the tokens, k the experts per
token, E the experts.  live is the number of tokens of a padded batch that are
real, off the share of experts that are switched off (logit -inf).
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the gate of a decode step (256 experts, 8 a token): latency
        {"name": "route_decode", "kind": "route", "T": 8, "E": 256, "k": 8, "score": "softmax", "dtype": "bf16",
         "bias": False, "groups": 1, "keep": 1, "top": 1, "renorm": True, "scale": 1.0, "live": 8, "off": 0.0},
        # a padded prefill chunk with a balance bias and groups of experts
        {"name": "route_prefill", "kind": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "dtype": "fp32",
         "bias": True, "groups": 8, "keep": 4, "top": 2, "renorm": True, "scale": 2.5, "live": 16101, "off": 0.0},
        # training: weights that are not renormalised, so every logit has a gradient; odd token count
        {"name": "route_backward_dense", "kind": "route_backward", "T": 4099, "E": 256, "k": 8, "score": "softmax",
         "dtype": "bf16", "renorm": False, "scale": 1.0, "off": 0.05},
        # training: renormalised sigmoids, where only the chosen logits have one
        {"name": "route_backward_chosen", "kind": "route_backward", "T": 16384, "E": 256, "k": 8, "score": "sigmoid",
         "dtype": "fp32", "renorm": True, "scale": 2.5, "off": 0.0},
        # one decode step's activations of a K = 5120 layer: latency
        {"name": "norm_decode", "kind": "norm", "M": 8, "K": 5120, "offset": 1.0, "residual": True},
        # a prefill chunk's
        {"name": "norm_prefill", "kind": "norm", "M": 8192, "K": 5120, "offset": 0.0, "residual": True},
        # the MLP's gate/up output ahead of the down projection, a decode batch
        {"name": "silu_decode", "kind": "silu", "M": 16, "K": 17408},
        # and a prefill chunk, odd row count
        {"name": "silu_prefill", "kind": "silu", "M": 4093, "K": 17408},
        # decode batch on the fused gate/up projection's half: weight stream
        {"name": "gemm_decode", "kind": "gemm", "M": 8, "N": 17408, "K": 5120},
        # the large prefill product: matrix cores, odd row count
        {"name": "gemm_prefill", "kind": "gemm", "M": 8191, "N": 10240, "K": 5120},
        # the experts' gate/up products in a decode step: few rows per expert
        {"name": "grouped_decode", "kind": "grouped", "T": 16, "k": 8, "E": 256, "N": 1024, "K": 2048},
        # and in prefill: a few hundred rows per expert, uneven
        {"name": "grouped_prefill", "kind": "grouped", "T": 8192, "k": 8, "E": 256, "N": 1024, "K": 2048},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["route", "route", "route_backward", "norm", "silu", "gemm", "gemm", "gemm", "grouped", "grouped"])
    if kind in ("route", "route_backward"):
        E = _logint(rng, 8, 512)
        T = _logint(rng, 1, min(16384, 16384 * 256 // E))
        k = rng.randint(1, min(E, 10))
        case = {"kind": kind, "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "dtype": rng.choice(["bf16", "fp32"]), "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 1.0, 2.5]),
                "off": rng.choice([0.0, 0.0, 0.1])}
        if kind == "route":
            groups = rng.choice([g for g in (1, 1, 1, 2, 3, 4, 8, 16) if E % g == 0])
            size = E // groups
            keep = rng.randint(-(-k // size), groups)
            case.update(bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]) if size >= 2 else 1,
                        live=T - (rng.randint(0, T // 8) if rng.random() < 0.3 else 0))
        return case
    if kind in ("norm", "silu"):
        K = 8 * _logint(rng, 4, 2176)
        limit = 8192 * 5120 if kind == "norm" else 4093 * 17408
        case = {"kind": kind, "M": min(_logint(rng, 1, 16384), limit // K), "K": K}
        if kind == "norm":
            case.update(offset=rng.choice([0.0, 1.0]), residual=rng.random() < 0.8)
        return case
    if kind == "gemm":
        N, K = _logint(rng, 16, 34816), 16 * _logint(rng, 4, 1088)
        if rng.random() < 0.7:
            N = (N + 15) // 16 * 16
        return {"kind": kind, "M": max(1, min(_logint(rng, 1, 8192), 8191 * 10240 * 5120 // (N * K))), "N": N, "K": K}
    k, E = rng.randint(1, 10), _logint(rng, 10, 512)
    N, K = 8 * _logint(rng, 8, 256), 16 * _logint(rng, 8, 256)
    E = max(10, min(E, 256 * 1024 * 2048 // (N * K)))
    T = max(1, min(_logint(rng, 1, 16384), 65536 * 1024 * 2048 // (k * N * K), 65536 // k))
    return {"kind": kind, "T": T, "k": k, "E": E, "N": N, "K": K}


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    kind = case["kind"]
    if kind == "route":
        T, E, k, live = case["T"], case["E"], case["k"], case["live"]
        return {"bytes": live * E * _size(case) + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 8 * live * E}
    if kind == "route_backward":
        T, E, k, b = case["T"], case["E"], case["k"], _size(case)
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * b + 8 * T * k + (T * E * b if dense else T * k * b),
                "flops": (8 * T * E if dense else 0) + 12 * T * k}
    if kind == "norm":
        M, n = case["M"], case["M"] * case["K"]
        # values (and the residual) in, the sum and the codes out; codes in, values out
        return {"bytes": (7 if case["residual"] else 3) * n + 2 * case["K"] + 8 * M + 3 * n, "flops": 10 * n}
    if kind == "silu":
        n = case["M"] * case["K"]
        return {"bytes": 5 * n + 3 * n + 8 * case["M"], "flops": 12 * n}
    N, K = case["N"], case["K"]
    if kind == "gemm":
        M = case["M"]
        return {"bytes": (M + N) * (K + 4) + 2 * M * N, "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    P = T * k
    active = E * (1.0 - (1.0 - min(1.0, k / E)) ** T)
    return {"bytes": int(active * N * (K + 4)) + T * (K + 4) + 2 * P * N + 4 * P + 4 * (E + 1), "flops": 2 * P * N * K}


# --------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std
    if outliers:
        x *= torch.where(torch.rand(shape, generator=gen, device="cuda") < outliers, 8.0, 1.0)
    return x.to(torch.bfloat16)


def _codes(x):
    """Stored int8 codes of bf16 rows and the scale of each row."""
    x = x.float()
    s = x.abs().amax(-1).clamp(min=1e-30) / 127.0
    return torch.round(x / s[..., None]).to(torch.int8), s


def _logits(gen, case):
    """The gate's output: some experts liked more, some switched off."""
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn((E,), generator=gen, device="cuda")
    if case["off"]:
        gone = torch.rand((E,), generator=gen, device="cuda") < case["off"]
        x = torch.where(gone, -math.inf, x)
    return x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)


def _sorted_slots(gen, T, k, E):
    """A routed batch in the order of the experts: (rows of the slots, offsets)."""
    score = torch.rand((T, E), generator=gen, device="cuda")
    if T >= 1024:
        score += 0.15 * torch.randn((E,), generator=gen, device="cuda")
    ids = torch.topk(score, k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0)
    return (order // k).to(torch.int32), offsets.to(torch.int32)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    if kind == "route":
        s = {"logits": _logits(gen, case), "bias": None, "rows": None}
        if case["bias"]:
            s["bias"] = 0.05 * torch.randn((case["E"],), generator=gen, device="cuda")
        if case["live"] < case["T"]:
            s["rows"] = torch.full((1,), case["live"], dtype=torch.int32, device="cuda")
        return s
    if kind == "route_backward":
        logits = _logits(gen, case)
        # the choice of the forward pass; -1 where fewer than k experts are on
        top = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        ids, vals = top.indices[:, :case["k"]], top.values[:, :case["k"]]
        ids = torch.where(vals == -math.inf, -1, ids).to(torch.int32).contiguous()
        return {"logits": logits, "ids": ids,
                "dweights": torch.randn((case["T"], case["k"]), generator=gen, device="cuda")}
    if kind == "norm":
        M, K = case["M"], case["K"]
        return {"y": _normal(gen, (M, K), 1.0, 0.001), "gamma": _normal(gen, (K,), 0.1),
                "residual": _normal(gen, (M, K), 2.0) if case["residual"] else None}
    if kind == "silu":
        return {"gu": _normal(gen, (case["M"], 2 * case["K"]), 1.0, 0.001)}
    N, K = case["N"], case["K"]
    if kind == "gemm":
        a, asc = _codes(_normal(gen, (case["M"], K), 1.0, 0.001))
        w, wsc = _codes(_normal(gen, (N, K), 0.02))
        return {"a": a, "asc": asc, "w": w, "wsc": wsc}
    E = case["E"]
    a, asc = _codes(_normal(gen, (case["T"], K), 1.0, 0.001))
    rows, offsets = _sorted_slots(gen, case["T"], case["k"], E)
    w = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    wsc = torch.empty((E, N), dtype=torch.float32, device="cuda")
    for e0 in range(0, E, 32):
        e1 = min(E, e0 + 32)
        w[e0:e1], wsc[e0:e1] = _codes(_normal(gen, (e1 - e0, N, K), 0.02))
    return {"a": a, "asc": asc, "w": w, "wsc": wsc, "rows": rows, "offsets": offsets}


def prepare(case, seed):
    s = _inputs(case, seed)
    kind = case["kind"]
    s["case"] = case
    if own:
        import block_scaled_precision_04_amd as bs
        s["bs"] = bs
        if kind in ("route", "route_backward"):
            s["score"] = bs.BS_SCORE_SOFTMAX if case["score"] == "softmax" else bs.BS_SCORE_SIGMOID
        if kind == "gemm":
            s["pre"], s["desc"] = bs.prelayout_int8(s.pop("w"))
            s["ws"] = bs.alloc_workspace(bs.BS_OP_W8A8_INT8, case["M"], case["N"], case["K"])
        if kind == "grouped":
            s["pre"], s["desc"] = bs.prelayout_int8_experts(s.pop("w"))
    elif kind == "grouped":
        s["bounds"] = s["offsets"].tolist()     # the plain loop over experts runs on host bounds
    return s


# ------------------------------------------------------------ the plain forms
def _plain_route(s):
    """Choices are decided next to borders: in 64 bits."""
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    x = s["logits"].double()
    masked = x == -math.inf
    if case["score"] == "softmax":
        ex = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        score = ex / ex.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    value = score if s["bias"] is None else score + s["bias"].double()
    value = torch.where(masked, -math.inf, value)
    if G > 1:
        by_group = value.reshape(T, G, E // G)
        best = torch.sort(by_group, dim=2, descending=True).values[:, :, :case["top"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        kept.scatter_(1, order[:, :case["keep"]], True)
        value = torch.where(kept[:, :, None], by_group, -math.inf).reshape(T, E)
    top = torch.sort(value, dim=1, descending=True, stable=True)
    ids = top.indices[:, :k]
    there = top.values[:, :k] > -math.inf
    there &= (torch.arange(T, device=x.device) < case["live"])[:, None]
    w = torch.where(there, torch.gather(score, 1, ids), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(there, ids, -1).to(torch.int32), (case["scale"] * w).float()


def _plain_route_backward(s):
    case = s["case"]
    x, g = s["logits"].float(), s["dweights"]
    ids = s["ids"].long()
    there = ids >= 0
    at = ids.clamp(min=0)
    g = torch.where(there, g, 0.0)
    if case["score"] == "softmax":
        ex = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e30))
        score = ex / ex.sum(1, keepdim=True).clamp(min=1e-38)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    sj = torch.where(there, torch.gather(score, 1, at), 0.0)
    d = torch.zeros_like(x)
    if case["renorm"]:
        p = sj / sj.sum(1, keepdim=True).clamp(min=1e-38)
        dj = case["scale"] * p * (g - (p * g).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            dj = dj * (1.0 - sj)
        d.scatter_add_(1, at, dj)
    elif case["score"] == "sigmoid":
        d.scatter_add_(1, at, case["scale"] * g * sj * (1.0 - sj))
    else:
        d.scatter_add_(1, at, g)
        d = case["scale"] * score * (d - (g * sj).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _plain_quant(h):
    """fp32 rows -> (the values of their int8 codes, bf16; the scales).  Codes are
    decided next to borders: quotients in 64 bits."""
    s = torch.clamp(h.abs().amax(1) / 127.0, min=2.0 ** -126)
    q = torch.round(h.double() / s.double()[:, None])
    return (q * s.double()[:, None]).to(torch.bfloat16), s


def _run_plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "route":
        return _plain_route(s)
    if kind == "route_backward":
        return _plain_route_backward(s)
    if kind == "norm":
        M, K = case["M"], case["K"]
        values = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        scale = torch.empty((M,), dtype=torch.float32, device="cuda")
        r = s["y"] if s["residual"] is None else (s["y"].float() + s["residual"].float()).to(torch.bfloat16)
        for m0 in range(0, M, 2048):
            d = r[m0:m0 + 2048].double()
            h = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6) * (case["offset"] + s["gamma"].double())
            values[m0:m0 + 2048], scale[m0:m0 + 2048] = _plain_quant(h.float())
        return (values, scale) if s["residual"] is None else (values, scale, r)
    if kind == "silu":
        M, K = case["M"], case["K"]
        values = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        scale = torch.empty((M,), dtype=torch.float32, device="cuda")
        for m0 in range(0, M, 1024):
            g, u = s["gu"][m0:m0 + 1024, :K].double(), s["gu"][m0:m0 + 1024, K:].double()
            values[m0:m0 + 1024], scale[m0:m0 + 1024] = _plain_quant((g / (1.0 + torch.exp(-g)) * u).float())
        return values, scale
    if kind == "gemm":
        return _plain_product(s["a"], s["w"], s["asc"], s["wsc"])
    out = torch.empty((case["T"] * case["k"], case["N"]), dtype=torch.bfloat16, device="cuda")
    for e, (r0, r1) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if r1 > r0:
            rows = s["rows"][r0:r1].long()
            out[r0:r1] = _plain_product(s["a"][rows], s["w"][e], s["asc"][rows], s["wsc"][e])
    return out


def _plain_product(a, w, asc, wsc):
    # sums of 1024 products are whole numbers below 2^24, exact in 32 bits; their sum is kept in 64
    acc = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    for k0 in range(0, a.shape[1], 1024):
        acc += a[:, k0:k0 + 1024].float() @ w[:, k0:k0 + 1024].float().t()
    return (acc * asc[:, None].double() * wsc.double()).to(torch.bfloat16)


def run(state):
    if not own:
        return _run_plain(state)
    s, bs, case = state, state["bs"], state["case"]
    kind = case["kind"]
    if kind == "route":
        return bs.moe_route(s["logits"], case["k"], bias=s["bias"], score=s["score"], groups=case["groups"],
                            topk_groups=case["keep"], group_top=case["top"], renorm=case["renorm"], scale=case["scale"],
                            rows=s["rows"])
    if kind == "route_backward":
        return bs.moe_route_backward(s["dweights"], s["logits"], s["ids"], score=s["score"], renorm=case["renorm"],
                                     scale=case["scale"])
    if kind == "norm":
        if s["residual"] is None:
            q, scale, _ = bs.add_rms_quant_int8(s["y"], None, s["gamma"], 1e-6, offset=case["offset"])
            return bs.dequant_int8(q, scale), scale
        q, scale, r = bs.add_rms_quant_int8(s["y"], s["residual"], s["gamma"], 1e-6, offset=case["offset"])
        return bs.dequant_int8(q, scale), scale, r
    if kind == "silu":
        q, scale = bs.silu_mul_quant_int8(s["gu"])
        return bs.dequant_int8(q, scale), scale
    if kind == "gemm":
        return bs.bsgemm_w8a8_int8(s["a"], s["asc"], s["desc"], s["pre"], s["wsc"], ws=s["ws"])
    return bs.bsgemm_w8a8_int8_grouped(s["a"], s["asc"], s["offsets"], s["desc"], s["pre"], s["wsc"], rows=s["rows"])


# ------------------------------------------------- the definitions in 64 bits
def _exact_best(value, n):
    """The n largest of each row, one after the other, ties to the lowest index;
    -1 where only -inf is left."""
    value = value.clone()
    index = torch.arange(value.shape[1], device=value.device)
    picks = []
    for _ in range(n):
        m = value.amax(1, keepdim=True)
        at = torch.where(value == m, index, value.shape[1]).amin(1)
        picks.append(torch.where(m[:, 0] == -math.inf, -1, at))
        value.scatter_(1, at[:, None], -math.inf)
    return torch.stack(picks, 1)


def _exact_scores(x, how):
    if how == "sigmoid":
        return torch.sigmoid(x)
    # (a token whose experts are all off has no scores)
    return torch.nan_to_num(torch.exp(x - torch.logsumexp(x, 1, keepdim=True)), nan=0.0)


def _exact_route(s, case):
    x = s["logits"].double()
    score = _exact_scores(x, case["score"])
    value = score + (0.0 if s["bias"] is None else s["bias"].double())
    value = value.masked_fill(torch.isinf(x), -math.inf)
    G, size = case["groups"], case["E"] // case["groups"]
    if G > 1:
        parts = torch.stack([torch.topk(value[:, i * size:(i + 1) * size], case["top"], dim=1).values.sum(1)
                             for i in range(G)], 1)
        # a group without enough experts that are on counts less than any other, but may be kept
        kept = _exact_best(torch.where(parts == -math.inf, -1e300, parts), case["keep"])
        keep = torch.zeros_like(parts)
        keep.scatter_(1, kept, 1.0)
        value = value.masked_fill(keep.repeat_interleave(size, 1) == 0, -math.inf)
    ids = _exact_best(value, case["k"])
    ids[case["live"]:] = -1
    w = torch.gather(score, 1, ids.clamp(min=0)) * (ids >= 0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return ids.to(torch.int32), case["scale"] * w


def _exact_route_backward(s, case):
    # dw_j / dl_e written out as a matrix, a run of tokens at a time
    x, E = s["logits"].double(), case["E"]
    out = torch.empty_like(x)
    for t0 in range(0, case["T"], 256):
        xs, ids = x[t0:t0 + 256], s["ids"][t0:t0 + 256].long()
        there = (ids >= 0).double()
        hot = torch.nn.functional.one_hot(ids.clamp(min=0), E).double() * there[:, :, None]      # [t, k, E]
        score = _exact_scores(xs, case["score"])
        sj = (hot * score[:, None, :]).sum(2)
        if case["score"] == "sigmoid":
            jac = hot * (score * (1.0 - score))[:, None, :]
        else:
            jac = sj[:, :, None] * (hot - score[:, None, :])
        if case["renorm"]:
            total = sj.sum(1).clamp(min=1e-300)[:, None, None]
            jac = (jac * total - sj[:, :, None] * jac.sum(1, keepdim=True)) / total ** 2
        out[t0:t0 + 256] = case["scale"] * (s["dweights"][t0:t0 + 256].double()[:, :, None] * jac).sum(1)
    return out


def _exact_quant(h):
    """fp64 rows that are fp32 values -> (values, scales): the nearest multiple of
    the scale, at the middle the even one."""
    scale = torch.clamp((h.abs().amax(1) / 127.0).to(torch.float32).double(), min=2.0 ** -126)
    t = h / scale[:, None]
    low = torch.floor(t)
    part = t - low
    up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return (low + up) * scale[:, None], scale


def exact(case, seed):
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "route":
        return _exact_route(s, case)
    if kind == "route_backward":
        return _exact_route_backward(s, case)
    if kind in ("norm", "silu"):
        M, K = case["M"], case["K"]
        values = torch.empty((M, K), dtype=torch.float64, device="cuda")
        scale = torch.empty((M,), dtype=torch.float64, device="cuda")
        total = torch.empty((M, K), dtype=torch.float64, device="cuda") if kind == "norm" else None
        for m0 in range(0, M, 512):
            m1 = min(M, m0 + 512)
            if kind == "norm":
                r = s["y"][m0:m1].double()
                if s["residual"] is not None:
                    r = (r + s["residual"][m0:m1].double()).to(torch.bfloat16).double()
                total[m0:m1] = r
                rms = torch.linalg.vector_norm(r, dim=1, keepdim=True).square() / K + 1e-6
                h = (r * torch.rsqrt(rms) * (s["gamma"].double() + case["offset"])).to(torch.float32)
            else:
                g, u = s["gu"][m0:m1, :K].double(), s["gu"][m0:m1, K:].double()
                h = (g * torch.sigmoid(g) * u).to(torch.float32)
            values[m0:m1], scale[m0:m1] = _exact_quant(h.double())
        if kind == "norm" and s["residual"] is not None:
            return values, scale, total
        return values, scale
    if kind == "gemm":
        return (s["a"].double() * s["asc"].double()[:, None]) @ (s["w"].double() * s["wsc"].double()[:, None]).t()
    bounds = s["offsets"].tolist()
    a = s["a"].double() * s["asc"].double()[:, None]
    out = torch.empty((case["T"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if bounds[e + 1] > bounds[e]:
            w = s["w"][e].double() * s["wsc"][e].double()[:, None]
            out[bounds[e]:bounds[e + 1]] = a[s["rows"][bounds[e]:bounds[e + 1]].long()] @ w.t()
    return out

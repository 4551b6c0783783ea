"""Cases that time the MXFP4 W4A4 and mixture-of-experts operators.

Every case runs one operator on inputs made from a seed.  With ``own`` false
the operator is computed in its plain form (elementary torch operations); with
``own`` true through the library's entry points, as a program would call them.

Kinds of case:
  quant    bf16 [M, K] -> MXFP4 (e2m1 codes, one e8m0 scale per 32) and read
           back as bf16, the values the codes stand for
  silu     the same from a gate/up projection's output [M, 2K]
  gemm     C = A . W^T, both operands MXFP4
  dispatch expert ids [T, k] -> sorted order, and the token rows in that order
  grouped  the experts' products on the sorted rows (rows read through the
           order, weights of all experts in one buffer)
  combine  the experts' outputs back in token order, weighted and summed
  combine_backward  the gradient of combine for the outputs and the weights

K is the inner size, N the output columns, T the tokens, k the experts per
token, E the experts, drop the share of (token, expert) pairs that belong to
no local expert (id -1, as on a rank that holds part of the experts).
"""
import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's activations of a K = 5120 layer: latency
        {"name": "quant_decode", "kind": "quant", "M": 8, "K": 5120},
        # a prefill chunk's activations
        {"name": "quant_prefill", "kind": "quant", "M": 8192, "K": 5120},
        # the MLP's gate/up output ahead of the down projection, odd row count
        {"name": "silu_prefill", "kind": "silu", "M": 4093, "K": 17408},
        # decode batch on the fused gate/up projection's half: weight stream
        {"name": "gemm_decode", "kind": "gemm", "M": 8, "N": 17408, "K": 5120},
        # a ragged mid-size batch (mixed prefill and decode)
        {"name": "gemm_ragged", "kind": "gemm", "M": 301, "N": 10240, "K": 5120},
        # the large prefill product: matrix cores
        {"name": "gemm_prefill", "kind": "gemm", "M": 8192, "N": 10240, "K": 5120},
        # decode batch through the MoE gate's experts (256 experts, hidden 2048)
        {"name": "dispatch_decode", "kind": "dispatch", "T": 8, "k": 8, "E": 256, "K": 2048, "drop": 0.0},
        # prefill on a rank that holds three quarters of the experts
        {"name": "dispatch_prefill", "kind": "dispatch", "T": 8192, "k": 8, "E": 256, "K": 2048, "drop": 0.25},
        # the experts' gate/up products in a decode step: few rows per expert
        {"name": "grouped_decode", "kind": "grouped", "T": 16, "k": 8, "E": 256, "N": 1024, "K": 2048, "drop": 0.0},
        # and in prefill: a few hundred rows per expert, uneven
        {"name": "grouped_prefill", "kind": "grouped", "T": 8192, "k": 8, "E": 256, "N": 1024, "K": 2048,
         "drop": 0.0},
        # a token's expert outputs summed back, odd token count
        {"name": "combine", "kind": "combine", "T": 4099, "k": 8, "E": 256, "K": 2048, "drop": 0.0},
        # its gradient, with dropped pairs
        {"name": "combine_backward", "kind": "combine_backward", "T": 8192, "k": 8, "E": 256, "K": 2048,
         "drop": 0.25},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["quant", "silu", "gemm", "gemm", "dispatch", "grouped", "grouped", "combine",
                       "combine_backward"])
    if kind in ("quant", "silu"):
        K = 32 * _logint(rng, 1, 544)
        limit = 8192 * 5120 if kind == "quant" else 4093 * 17408
        return {"kind": kind, "M": min(_logint(rng, 1, 16384), limit // K), "K": K}
    if kind == "gemm":
        N, K = 16 * _logint(rng, 1, 2176), 128 * _logint(rng, 1, 136)
        return {"kind": kind, "M": max(1, min(_logint(rng, 1, 8192), 8192 * 10240 * 5120 // (N * K))), "N": N, "K": K}
    k, E = rng.randint(1, 10), _logint(rng, 10, 512)
    drop = rng.choice([0.0, 0.0, 0.3])
    if kind == "grouped":
        N, K = 16 * _logint(rng, 4, 128), 128 * _logint(rng, 1, 32)
        E = max(10, min(E, 256 * 1024 * 2048 // (N * K)))
        T = max(1, min(_logint(rng, 1, 16384), 65536 * 1024 * 2048 // (k * N * K), 65536 // k))
        return {"kind": kind, "T": T, "k": k, "E": E, "N": N, "K": K, "drop": drop}
    K = 8 * _logint(rng, 1, 640)
    T = max(1, min(_logint(rng, 1, 16384), 65536 * 2048 // (k * K), 65536 // k))
    return {"kind": kind, "T": T, "k": k, "E": E, "K": K, "drop": drop}


def _pairs(case):
    return int(case["T"] * case["k"] * (1.0 - case["drop"]))


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    kind = case["kind"]
    if kind in ("quant", "silu"):
        n = case["M"] * case["K"]
        code = n // 2 + n // 32
        # values in, codes out, codes in, values out
        return {"bytes": (2 if kind == "quant" else 4) * n + 2 * code + 2 * n, "flops": (4 if kind == "quant" else 12) * n}
    if kind == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K // 2 + K // 32) + 2 * M * N, "flops": 2 * M * N * K}
    T, k, E, K, P = case["T"], case["k"], case["E"], case["K"], _pairs(case)
    if kind == "dispatch":
        return {"bytes": 3 * 4 * T * k + 4 * (E + 1) + 2 * T * K + 2 * P * K, "flops": 0}
    if kind == "grouped":
        N = case["N"]
        active = E * (1.0 - (1.0 - k * (1.0 - case["drop"]) / E) ** T)
        return {"bytes": int(active * N * (K // 2 + K // 32)) + min(T, P) * (K // 2 + K // 32) + 2 * P * N + 4 * P,
                "flops": 2 * P * N * K}
    if kind == "combine":
        return {"bytes": 2 * P * K + 2 * T * K + 8 * T * k, "flops": 2 * P * K}
    return {"bytes": 4 * P * K + 2 * T * K + 12 * T * k, "flops": 3 * P * K}


# --------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std
    if outliers:
        x *= torch.where(torch.rand(shape, generator=gen, device="cuda") < outliers, 8.0, 1.0)
    return x.to(torch.bfloat16)


def _pack(x):
    """MXFP4 of bf16 rows as stored bytes: packed codes [.., K/2], e8m0 [.., K/32]."""
    *lead, K = x.shape
    b = x.float().reshape(*lead, K // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.clamp(torch.frexp(amax)[1] - 3, min=-127)
    t = torch.ldexp(b, -e)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    t_abs = t.abs().contiguous()
    lo = torch.bucketize(t_abs, mids)                   # a midpoint goes down
    hi = torch.bucketize(t_abs, mids, right=True)       # a midpoint goes up
    code = torch.where(lo % 2 == 0, lo, hi).to(torch.uint8)
    code |= torch.where(torch.signbit(t), 8, 0).to(torch.uint8)
    code = code.reshape(*lead, K // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), (e.squeeze(-1) + 127).to(torch.uint8).contiguous()


def _ids(gen, case):
    """Expert ids [T, k]: k different experts a token, some experts liked more in
    large batches; a share of the pairs dropped."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.rand((T, E), generator=gen, device="cuda")
    if T >= 1024:
        score += 0.15 * torch.randn((E,), generator=gen, device="cuda")
    ids = torch.topk(score, k, dim=1).indices.to(torch.int32)
    if case["drop"]:
        gone = torch.rand((T, k), generator=gen, device="cuda") < case["drop"]
        ids = torch.where(gone, -1, ids)
    return ids.contiguous()


def _order(ids, E):
    """(rows, pos, offsets) of a stable sort of the pairs by expert id."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    ends = torch.cumsum(counts, 0)
    total = ends[E - 1]
    slot = torch.arange(T * k, device=ids.device)
    rows = torch.where(slot < total, order // k, -1)
    pos = torch.empty_like(slot)
    pos[order] = torch.where(slot < total, slot, -1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = ends[:E].to(torch.int32)
    return rows.to(torch.int32), pos.to(torch.int32).reshape(T, k), offsets


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, K = case["kind"], case["K"]
    if kind == "quant":
        return {"x": _normal(gen, (case["M"], K), 1.0, 0.001)}
    if kind == "silu":
        return {"gu": _normal(gen, (case["M"], 2 * K), 1.0, 0.001)}
    if kind == "gemm":
        a, asc = _pack(_normal(gen, (case["M"], K), 1.0, 0.001))
        w, wsc = _pack(_normal(gen, (case["N"], K), 0.02))
        return {"a": a, "asc": asc, "w": w, "wsc": wsc}
    ids = _ids(gen, case)
    T, k, E = case["T"], case["k"], case["E"]
    if kind == "dispatch":
        return {"ids": ids, "x": _normal(gen, (T, K))}
    rows, pos, offsets = _order(ids, E)
    if kind == "grouped":
        a, asc = _pack(_normal(gen, (T, K), 1.0, 0.001))
        w = torch.empty((E, case["N"], K // 2), dtype=torch.uint8, device="cuda")
        wsc = torch.empty((E, case["N"], K // 32), dtype=torch.uint8, device="cuda")
        for e0 in range(0, E, 32):
            e1 = min(E, e0 + 32)
            w[e0:e1], wsc[e0:e1] = _pack(_normal(gen, (e1 - e0, case["N"], K), 0.02))
        return {"a": a, "asc": asc, "w": w, "wsc": wsc, "rows": rows, "offsets": offsets}
    g = torch.rand((T, k), generator=gen, device="cuda") + 0.05
    s = {"y": _normal(gen, (T * k, K)), "pos": pos, "weights": g / g.sum(1, keepdim=True)}
    if kind == "combine_backward":
        s["dout"] = _normal(gen, (T, K))
        s["used"] = (torch.arange(T * k, device="cuda") < offsets[E])[:, None]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    kind = case["kind"]
    s["case"] = case
    if kind == "dispatch":
        s["xs"] = torch.zeros((case["T"] * case["k"], case["K"]), dtype=torch.bfloat16, device="cuda")
    if kind == "grouped":
        s["out"] = torch.zeros((case["T"] * case["k"], case["N"]), dtype=torch.bfloat16, device="cuda")
    if kind == "combine_backward":
        s["dy"] = torch.zeros_like(s["y"])
    if own:
        import block_scaled_precision_04_amd as bs
        s["bs"] = bs
        if kind == "gemm":
            s["pre"], s["desc"] = bs.prelayout_mxfp4(s.pop("w"), s.pop("wsc"))
            s["ws"] = bs.alloc_workspace(bs.BS_OP_W4A4_MXFP4, case["M"], case["N"], case["K"])
        if kind == "grouped":
            s["pre"], s["desc"] = bs.prelayout_mxfp4_experts(s.pop("w"), s.pop("wsc"))
        if kind == "dispatch":
            s["ws"] = bs.alloc_workspace(bs.BS_OP_MOE_SORT, case["T"], case["k"], case["E"])
    elif kind == "grouped":
        s["bounds"] = s["offsets"].tolist()     # the plain loop over experts runs on host bounds
    return s


# ------------------------------------------------------------ the plain forms
def _round_trip(x):
    """Values that the MXFP4 codes of fp32 rows stand for, bf16."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.clamp(torch.frexp(amax)[1] - 3, min=-127)    # frexp's exponent is floor(log2) + 1
    t = torch.ldexp(b, -e)
    step = torch.exp2(torch.clamp(torch.frexp(t)[1] - 2, min=-1, max=1).float())
    t = torch.clamp(torch.round(t / step) * step, -6.0, 6.0)
    return torch.ldexp(t, e).reshape(x.shape).to(torch.bfloat16)


def _dequant(codes, scales):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.reshape(*scales.shape, 32) * torch.exp2(scales.float() - 127.0)[..., None]
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _run_plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "quant":
        return _round_trip(s["x"].float())
    if kind == "silu":
        # codes are decided next to borders: the product in 64 bits, rounded once to fp32
        K = case["K"]
        h = torch.empty((case["M"], K), dtype=torch.float32, device="cuda")
        for m0 in range(0, case["M"], 1024):
            g, u = s["gu"][m0:m0 + 1024, :K].double(), s["gu"][m0:m0 + 1024, K:].double()
            h[m0:m0 + 1024] = g / (1.0 + torch.exp(-g)) * u
        return _round_trip(h)
    if kind == "gemm":
        return (_dequant(s["a"], s["asc"]) @ _dequant(s["w"], s["wsc"]).t()).to(torch.bfloat16)
    if kind == "dispatch":
        rows, pos, offsets = _order(s["ids"], case["E"])
        keep = (rows >= 0)[:, None]
        return rows, pos, offsets, torch.where(keep, s["x"][rows.clamp(min=0).long()], s["xs"])
    if kind == "grouped":
        a = _dequant(s["a"], s["asc"])
        out = s["out"].clone()
        for e, (r0, r1) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if r1 > r0:
                rows = s["rows"][r0:r1].long()
                out[r0:r1] = (a[rows] @ _dequant(s["w"][e], s["wsc"][e]).t()).to(torch.bfloat16)
        return out
    pos = s["pos"].long()
    kept = pos >= 0
    at = pos.clamp(min=0)
    w = torch.where(kept, s["weights"], 0.0)
    if kind == "combine":
        out = torch.zeros((case["T"], case["K"]), dtype=torch.float32, device="cuda")
        for j in range(case["k"]):
            out += w[:, j, None] * s["y"][at[:, j]].float()
        return out.to(torch.bfloat16)
    dout = s["dout"].float()
    dw = torch.empty_like(s["weights"])
    src = torch.zeros(case["T"] * case["k"] + 1, dtype=torch.long, device="cuda")
    src[torch.where(kept, pos, case["T"] * case["k"]).reshape(-1)] = torch.arange(pos.numel(), device="cuda")
    src = src[:-1]
    dy = (w.reshape(-1)[src][:, None] * dout[src // case["k"]]).to(torch.bfloat16)
    dy = torch.where(s["used"], dy, s["dy"])
    for j in range(case["k"]):
        dw[:, j] = torch.where(kept[:, j], (dout * s["y"][at[:, j]].float()).sum(1), 0.0)
    return dy, dw


def run(state):
    if not own:
        return _run_plain(state)
    s, bs, case = state, state["bs"], state["case"]
    kind = case["kind"]
    if kind == "quant":
        q, e = bs.quant_mxfp4(s["x"])
        return bs.dequant_mxfp4(q, e)
    if kind == "silu":
        q, e = bs.silu_mul_quant_mxfp4(s["gu"])
        return bs.dequant_mxfp4(q, e)
    if kind == "gemm":
        return bs.bsgemm_w4a4_mxfp4(s["a"], s["asc"], s["desc"], s["pre"], ws=s["ws"])
    if kind == "dispatch":
        rows, pos, offsets = bs.moe_sort(s["ids"], case["E"], ws=s["ws"])
        return rows, pos, offsets, bs.moe_gather(s["x"], pos, out=s["xs"])
    if kind == "grouped":
        return bs.bsgemm_w4a4_mxfp4_grouped(s["a"], s["asc"], s["offsets"], s["desc"], s["pre"], rows=s["rows"],
                                            out=s["out"])
    if kind == "combine":
        return bs.moe_combine(s["y"], s["pos"], s["weights"])
    return bs.moe_combine_backward(s["dout"], s["y"], s["pos"], s["weights"], dy=s["dy"])


# ------------------------------------------------- the definitions in 64 bits
def _exact_values(codes, scales):
    """MXFP4 bytes -> float64 values, from the format's bit fields."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).long()
    ex, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(ex == 0, man * 0.5, (1.0 + 0.5 * man) * torch.pow(2.0, (ex - 1).double()))
    v = torch.where(c >= 8, -mag, mag)
    return v * torch.pow(2.0, scales.double() - 127.0).repeat_interleave(32, -1)


def _exact_round_trip(x):
    """The MXFP4 round trip of float64 values: nearest of the format's values,
    ties to the even code."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    e = torch.where(torch.pow(2.0, e) > amax, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= amax, e + 1, e)
    scale = torch.pow(2.0, torch.clamp(e - 2, min=-127.0))
    scale = torch.where(amax > 0, scale, 1.0)
    t = b.abs() / scale
    out = torch.zeros_like(t)
    for i in range(1, 8):
        mid = 0.5 * (_E2M1[i - 1] + _E2M1[i])
        up = t > mid if i % 2 else t >= mid     # at the midpoint the even code wins
        out = torch.where(up, _E2M1[i], out)
    return (torch.sign(b) * out * scale).reshape(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "quant":
        return _exact_round_trip(s["x"].double())
    if kind == "silu":
        out = torch.empty((case["M"], case["K"]), dtype=torch.float64, device="cuda")
        for m0 in range(0, case["M"], 512):
            gu = s["gu"][m0:m0 + 512].double()
            g, u = gu[:, :case["K"]], gu[:, case["K"]:]
            h = (g * torch.sigmoid(g) * u).to(torch.float32).double()
            out[m0:m0 + 512] = _exact_round_trip(h)
        return out
    if kind == "gemm":
        return _exact_values(s["a"], s["asc"]) @ _exact_values(s["w"], s["wsc"]).t().contiguous()
    if kind == "dispatch":
        T, k, E, K = case["T"], case["k"], case["E"], case["K"]
        ids = s["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(E)]
        for p, e in enumerate(ids):
            if 0 <= e < E:
                lists[e].append(p)
        rows, pos, offsets = [-1] * (T * k), [-1] * (T * k), [0]
        slot = 0
        for pairs in lists:
            for p in pairs:
                rows[slot], pos[p] = p // k, slot
                slot += 1
            offsets.append(slot)
        xs = torch.zeros((T * k, K), dtype=torch.float64, device="cuda")
        xs[:slot] = s["x"].double()[torch.tensor(rows[:slot], device="cuda", dtype=torch.long)]
        as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        return as_int(rows), as_int(pos).reshape(T, k), as_int(offsets), xs
    if kind == "grouped":
        bounds = s["offsets"].tolist()
        out = torch.zeros((case["T"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
        a = _exact_values(s["a"], s["asc"])
        for e in range(case["E"]):
            if bounds[e + 1] > bounds[e]:
                w = _exact_values(s["w"][e], s["wsc"][e]).t().contiguous()
                out[bounds[e]:bounds[e + 1]] = a[s["rows"][bounds[e]:bounds[e + 1]].long()] @ w
        return out
    T, k, K = case["T"], case["k"], case["K"]
    pos, weights = s["pos"].long(), s["weights"].double()
    if kind == "combine":
        out = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(pos[:, j] >= 0).squeeze(1)
            out[t] += weights[t, j, None] * s["y"][pos[t, j]].double()
        return out
    dy = torch.zeros((T * k, K), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    dout = s["dout"].double()
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0).squeeze(1)
        dy[pos[t, j]] = weights[t, j, None] * dout[t]
        dw[t, j] = (dout[t] * s["y"][pos[t, j]].double()).sum(1)
    return dy, dw

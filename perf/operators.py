"""The FP8 (E4M3, one scale per block of 128) operators: what is measured, on which sizes.

Operators, by a case's ``op``:

- ``quant``: BF16 rows to E4M3 with one FP32 scale per row and 128 columns.
- ``dense``: product of quantised rows with an E4M3 weight that has one FP32 scale per
  128 x 128 block (the shared expert's down projection).
- ``dense_swiglu``: the shared expert's gate and up products, the clamped SwiGLU and the
  quantisation of its output.
- ``grouped``: the product grouped by expert over the expert-sorted slots (down projection).
- ``grouped_swiglu``: the same over the fused gate_up weight, rows gathered by token, with
  the clamped SwiGLU and the quantisation of its output.

Where ``own`` is false, ``run`` computes them with elementary torch operations in FP32;
where it is true, through ``grouped_nvfp4_w4a16_amd``.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126
LIMIT = 7.0  # the SwiGLU clamp of every workload in this repository


def listed():
    return [
        # Eight decode rows of the large configuration: a latency-bound step.
        {"name": "quant_decode", "op": "quant", "rows": 8, "cols": 6144},
        # Sixteen prefill sub-chunks' hidden states, once per layer.
        {"name": "quant_prefill", "op": "quant", "rows": 4096, "cols": 6144},
        # The shared expert's down projection for a single token.
        {"name": "dense_token", "op": "dense", "m": 1, "n": 6144, "k": 2048},
        # The same for one 256-row prefill sub-chunk, and for a long prompt.
        {"name": "dense_chunk", "op": "dense", "m": 256, "n": 6144, "k": 2048},
        {"name": "dense_long", "op": "dense", "m": 4096, "n": 6144, "k": 2048},
        # The shared expert's gate and up of a sub-chunk.
        {"name": "dense_swiglu_chunk", "op": "dense_swiglu", "m": 256, "n": 2048, "k": 6144},
        # A ragged verify batch on sizes no tile divides (partial scale blocks on each axis).
        {"name": "dense_swiglu_ragged", "op": "dense_swiglu", "m": 77, "n": 1360, "k": 1040},
        # Eight decode rows: 64 slots over about 57 of 256 experts, a few rows each.
        {"name": "grouped_decode", "op": "grouped", "rows": 8, "experts": 256, "top_k": 8,
         "n": 6144, "k": 2048, "zipf": 0.0},
        # One prefill sub-chunk: every expert's weights, about eight rows each.
        {"name": "grouped_chunk", "op": "grouped", "rows": 256, "experts": 256, "top_k": 8,
         "n": 6144, "k": 2048, "zipf": 0.0},
        {"name": "grouped_swiglu_chunk", "op": "grouped_swiglu", "rows": 256, "experts": 256,
         "top_k": 8, "n": 2048, "k": 6144, "zipf": 0.0},
        # The small layer under skewed routing: a few hot experts, several with no row.
        {"name": "grouped_swiglu_zipf", "op": "grouped_swiglu", "rows": 1001, "experts": 64,
         "top_k": 8, "n": 768, "k": 2048, "zipf": 1.1},
        # A long prompt in one call: about 128 rows per expert.
        {"name": "grouped_swiglu_long", "op": "grouped_swiglu", "rows": 4096, "experts": 256,
         "top_k": 8, "n": 2048, "k": 6144, "zipf": 0.0},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["quant", "dense", "dense_swiglu", "grouped", "grouped_swiglu"])
    if op == "quant":
        return {"op": op, "rows": _log_int(rng, 1, 4096), "cols": _log_int(rng, 128, 6144, 16)}
    if op in ("dense", "dense_swiglu"):
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 128, 6144, 16),
                "k": _log_int(rng, 128, 6144, 16)}
    top_k = rng.choice([1, 2, 4, 6, 8])
    experts = _log_int(rng, 8, 128)
    zipf = rng.choice([0.0, 0.0, 1.1])
    return {"op": op, "rows": _log_int(rng, 1, 1024), "experts": experts,
            "top_k": min(top_k, experts), "n": _log_int(rng, 128, 2048, 16),
            "k": _log_int(rng, 256, 4096, 16), "zipf": zipf}


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------ inputs


def _hidden(gen, rows, cols):
    """BF16 hidden states: normal, one channel in 256 an outlier."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x[:, 5::256] *= 16.0
    return x.to(torch.bfloat16)


def _codes(values, scale):
    return (values / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quantised_rows(gen, rows, cols):
    """Quantised rows as the step before the product leaves them."""
    x = _hidden(gen, rows, cols).float()
    pad = torch.nn.functional.pad(x, (0, _blocks(cols) * BLOCK - cols))
    amax = pad.view(rows, -1, BLOCK).abs().amax(2)
    scale = (amax / E4M3_MAX).clamp(min=MIN_SCALE)
    return _codes(x, scale.repeat_interleave(BLOCK, 1)[:, :cols]), scale


def _weights(gen, experts, n, k):
    """E4M3 weights [experts, n, k] of N(0, 1 / k) and their scales per 128 x 128 block."""
    nb, kb = _blocks(n), _blocks(k)
    w = torch.empty((experts, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((experts, nb, kb), dtype=torch.float32, device="cuda")
    step = max(1, min(experts, (1 << 28) // (n * k)))
    for e in range(0, experts, step):
        c = min(step, experts - e)
        v = torch.zeros((c, nb * BLOCK, kb * BLOCK), device="cuda")
        v[:, :n, :k] = torch.randn((c, n, k), generator=gen, device="cuda") / math.sqrt(k)
        b = v.view(c, nb, BLOCK, kb, BLOCK)
        s[e:e + c] = b.abs().amax((2, 4)) / E4M3_MAX
        q = _codes(b, s[e:e + c, :, None, :, None]).view(c, nb * BLOCK, kb * BLOCK)
        w[e:e + c] = q[:, :n, :k]
    return w, s


def _route(gen, rows, experts, top_k, zipf):
    """Expert-sorted slots: token of each sorted slot, offsets per expert, and the largest
    number of rows an expert has."""
    u = torch.rand((rows, experts), generator=gen, device="cuda", dtype=torch.float64)
    logits = -torch.log(-torch.log(u.clamp(1e-300, 1.0 - 1e-16)))
    rank = torch.randperm(experts, generator=gen, device="cuda") + 1
    ids = (logits - zipf * rank.double().log()).topk(top_k, dim=1).indices.view(-1)
    order = torch.argsort(ids, stable=True)
    count = torch.bincount(ids, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = count.cumsum(0)
    return (order // top_k).int(), offsets, int(count.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    st = {"op": op}
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        st["x"] = _hidden(gen, rows, cols)
        st["q"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
        st["scale"] = torch.empty((rows, _blocks(cols)), device="cuda")
        return st
    n, k = case["n"], case["k"]
    swiglu = op.endswith("swiglu")
    if op.startswith("dense"):
        rows = case["m"]
        st["a"], st["sa"] = _quantised_rows(gen, rows, k)
        w, s = _weights(gen, 2 if swiglu else 1, n, k)  # gate and up: two weights
        st["w"], st["sw"] = w, s
    else:
        experts, top_k = case["experts"], case["top_k"]
        rows = case["rows"] * top_k
        tok, st["offsets"], st["most"] = _route(gen, case["rows"], experts, top_k, case["zipf"])
        # gate_up gathers token rows; the down projection reads one row per sorted slot
        st["gather"] = tok if swiglu else None
        st["a"], st["sa"] = _quantised_rows(gen, case["rows"] if swiglu else rows, k)
        if swiglu:
            gate, sg = _weights(gen, experts, n, k)
            up, su = _weights(gen, experts, n, k)
            st["w"], st["sw"] = torch.cat((gate, up), 1), torch.cat((sg, su), 1)
            del gate, up
        else:
            st["w"], st["sw"] = _weights(gen, experts, n, k)
    if swiglu:
        st["q"] = torch.empty((rows, n), dtype=torch.float8_e4m3fn, device="cuda")
        st["scale"] = torch.empty((rows, _blocks(n)), device="cuda")
    else:
        st["c"] = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    if own and op.startswith("grouped"):
        import grouped_nvfp4_w4a16_amd as hip

        st["table"] = hip.Fp8ExpertTable(list(st["w"].unbind(0)), list(st["sw"].unbind(0)),
                                         st["w"].shape[1], k, gate_up=swiglu)
    return st


# ------------------------------------------------------------------- the operators, plain


def _rows_f32(codes, scale):
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _weight_f32(codes, scale):
    """[.., n, k] codes times their block scales [.., n / 128, k / 128]."""
    n, k = codes.shape[-2:]
    s = scale.repeat_interleave(BLOCK, -1)[..., :k]
    row = torch.arange(n, device=codes.device) // BLOCK
    return codes.float().mul_(s.index_select(-2, row))


def _quantise(v):
    rows, cols = v.shape
    pad = torch.nn.functional.pad(v, (0, _blocks(cols) * BLOCK - cols))
    scale = (pad.view(rows, -1, BLOCK).abs().amax(2) / E4M3_MAX).clamp(min=MIN_SCALE)
    q = v / scale.repeat_interleave(BLOCK, 1)[:, :cols]
    return q.to(torch.float8_e4m3fn), scale


def _swiglu(g, u):
    g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    return g / (1.0 + torch.exp(-g)) * u


def _grouped(x, w, offsets, most):
    """x [slots, k] in sorted order times each slot's expert's w [experts, n, k]: one
    batched product over the experts' rows, padded to the largest count."""
    slots = x.shape[0]
    at = offsets[:-1, None].long() + torch.arange(most, device=x.device)
    rows = x[at.clamp(max=slots - 1)] * (at < offsets[1:, None])[..., None]
    y = torch.bmm(w, rows.transpose(1, 2).contiguous())  # [experts, n, most]
    slot = torch.arange(slots, device=x.device)
    e = torch.searchsorted(offsets[1:].long().contiguous(), slot, right=True)
    return y.transpose(1, 2)[e, slot - offsets[e].long()]


def _plain(st):
    op = st["op"]
    if op == "quant":
        return list(_quantise(st["x"].float()))
    x = _rows_f32(st["a"], st["sa"])
    if op == "dense":
        return [(x @ _weight_f32(st["w"], st["sw"])[0].t()).to(torch.bfloat16)]
    if op == "dense_swiglu":
        w = _weight_f32(st["w"], st["sw"])
        return list(_quantise(_swiglu(x @ w[0].t(), x @ w[1].t())))
    if op == "grouped":
        y = _grouped(x, _weight_f32(st["w"], st["sw"]), st["offsets"], st["most"])
        return [y.to(torch.bfloat16)]
    experts, n2, k = st["w"].shape
    halves = st["w"].view(experts, 2, n2 // 2, k)
    w = _weight_f32(halves, st["sw"].view(experts, 2, -1, st["sw"].shape[2]))
    y = _grouped(x[st["gather"].long()], w.view(experts, n2, k), st["offsets"], st["most"])
    return list(_quantise(_swiglu(y[:, :n2 // 2], y[:, n2 // 2:])))


def _hip(st):
    import grouped_nvfp4_w4a16_amd as hip

    op = st["op"]
    if op == "quant":
        hip.moe_quant_fp8(st["x"], st["q"], st["scale"])
        return [st["q"], st["scale"]]
    if op == "dense":
        hip.moe_dense_gemm_fp8(st["a"], st["sa"], st["w"][0], st["sw"][0], st["c"])
        return [st["c"]]
    if op == "dense_swiglu":
        hip.moe_dense_gate_up_swiglu_fp8(st["a"], st["sa"], st["w"][0], st["sw"][0], st["w"][1],
                                         st["sw"][1], st["q"], st["scale"], LIMIT)
        return [st["q"], st["scale"]]
    if op == "grouped":
        hip.moe_w8a8_grouped_gemm(st["a"], st["sa"], st["table"], st["offsets"], st["c"])
        return [st["c"]]
    hip.moe_w8a8_grouped_gemm_swiglu(st["a"], st["sa"], st["table"], st["offsets"], st["q"],
                                     st["scale"], LIMIT, a_gather=st["gather"])
    return [st["q"], st["scale"]]


def run(state):
    return _hip(state) if own else _plain(state)


# ------------------------------------------------------------------------- work and exact


def _experts_used(case):
    """How many experts one routing of this kind reaches (a fixed sample of it)."""
    r = np.random.default_rng(1)
    logits = r.gumbel(size=(case["rows"], case["experts"]))
    logits -= case["zipf"] * np.log(np.arange(1, case["experts"] + 1))
    ids = np.argpartition(-logits, case["top_k"] - 1, axis=1)[:, :case["top_k"]]
    return len(np.unique(ids))


def work(case):
    op = case["op"]
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        # the absolute maximum, the division and the rounding: about four per value
        return {"bytes": rows * (3 * cols + 4 * _blocks(cols)), "flops": 4 * rows * cols}
    n, k = case["n"], case["k"]
    swiglu = op.endswith("swiglu")
    n_w = 2 * n if swiglu else n
    weight = n_w * k + 4 * (n_w // n) * _blocks(n) * _blocks(k)
    if op.startswith("dense"):
        rows = rows_in = case["m"]
        w_bytes = weight
        index = 0
    else:
        rows = case["rows"] * case["top_k"]
        rows_in = case["rows"] if swiglu else rows
        w_bytes = _experts_used(case) * weight
        index = 4 * (case["experts"] + 1) + (4 * rows if swiglu else 0)
    out = rows * (n + 4 * _blocks(n)) if swiglu else 2 * rows * n
    return {"bytes": w_bytes + rows_in * (k + 4 * _blocks(k)) + out + index,
            "flops": 2 * rows * n_w * k}


def _round_e4m3(v):
    """FP64 values to the nearest E4M3 value (ties to even), |v| <= 448 after rounding."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    ulp = torch.exp2(torch.clamp(e.double() - 1.0, min=-6.0) - 3.0)
    return torch.round(v / ulp) * ulp


def _exact_quantise(v):
    q, s = torch.empty_like(v), v.new_empty(v.shape[0], _blocks(v.shape[1]))
    for b in range(s.shape[1]):
        c = slice(b * BLOCK, min((b + 1) * BLOCK, v.shape[1]))
        s[:, b] = torch.clamp(v[:, c].abs().max(dim=1).values / E4M3_MAX, min=MIN_SCALE)
        q[:, c] = _round_e4m3(v[:, c] / s[:, b:b + 1])
    return [q, s]


def _exact_product(a, sa, w, sw):
    """sum over the blocks of 128 k of (codes product) * row scale * block scale, FP64."""
    n, k = w.shape
    rows_n = torch.arange(n, device=w.device) // BLOCK
    y = torch.zeros((a.shape[0], n), dtype=torch.float64, device=w.device)
    for b in range(_blocks(k)):
        c = slice(b * BLOCK, min((b + 1) * BLOCK, k))
        part = a[:, c].double() @ w[:, c].double().t()
        y += part * sa[:, b:b + 1].double() * sw[rows_n, b].double()
    return y


def _exact_swiglu(g, u):
    g = torch.minimum(g, torch.full_like(g, LIMIT))
    u = torch.maximum(torch.minimum(u, torch.full_like(u, LIMIT)), torch.full_like(u, -LIMIT))
    return g * torch.sigmoid(g) * u


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _exact_quantise(st["x"].double())
    a, sa, w, sw = st["a"], st["sa"], st["w"], st["sw"]
    if op == "dense":
        return [_exact_product(a, sa, w[0], sw[0])]
    if op == "dense_swiglu":
        return _exact_quantise(_exact_swiglu(_exact_product(a, sa, w[0], sw[0]),
                                             _exact_product(a, sa, w[1], sw[1])))
    n, nb = case["n"], _blocks(case["n"])
    bounds = st["offsets"].tolist()
    out = []
    for e in range(case["experts"]):
        s = slice(bounds[e], bounds[e + 1])
        if s.start == s.stop:
            continue
        if op == "grouped":
            out.append(_exact_product(a[s], sa[s], w[e], sw[e]))
            continue
        t = st["gather"][s].long()
        out.append(_exact_swiglu(_exact_product(a[t], sa[t], w[e, :n], sw[e, :nb]),
                                 _exact_product(a[t], sa[t], w[e, n:], sw[e, nb:])))
    y = torch.cat(out)
    return [y] if op == "grouped" else _exact_quantise(y)

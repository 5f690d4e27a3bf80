"""The feed-forward half of a decoder layer around the routed experts: what is measured.

Operators, by a case's ``op``:

- ``norm``: the residual's addition, the root-mean-square norm, and its output both in BF16
  (the router and the BF16 experts read it) and in E4M3 with one FP32 scale per 128 columns
  (the FP8 experts read it).
- ``dense_int8``: product of INT8 rows (one scale per token) with an INT8 weight (one scale per
  output channel), BF16 out.
- ``swiglu_int8``: the gate and up products in INT8 and the clamped SwiGLU, BF16 out.
- ``mlp_int8``: residual + norm with an INT8 output, then the whole shared expert in INT8 (gate,
  up, SwiGLU, quantisation, down): the operators in the order a layer calls them.
- ``few``: a whole routed NVFP4 layer for a few tokens, from the router's logits to the weighted
  sum of the experts' outputs and the shared expert's term.

Where ``own`` is false, ``run`` computes them with elementary torch operations in FP32; where it
is true, through ``grouped_nvfp4_w4a16_amd``.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 128  # columns per scale of the E4M3 output
E4M3_MAX = 448.0
INT8_MAX = 127.0
MIN_SCALE = 2.0 ** -126
LIMIT = 7.0  # the SwiGLU clamp of every workload in this repository
EPS = 1e-6


def listed():
    return [
        # Eight decode rows of the large configuration: a latency-bound step.
        {"name": "norm_decode", "op": "norm", "rows": 8, "cols": 6144},
        # Sixteen prefill sub-chunks' hidden states, once per layer.
        {"name": "norm_prefill", "op": "norm", "rows": 4096, "cols": 6144},
        # The shared expert's down projection for a single token.
        {"name": "dense_int8_token", "op": "dense_int8", "m": 1, "n": 6144, "k": 2048},
        # The same for one 256-row prefill sub-chunk, and for a long prompt.
        {"name": "dense_int8_chunk", "op": "dense_int8", "m": 256, "n": 6144, "k": 2048},
        {"name": "dense_int8_long", "op": "dense_int8", "m": 4096, "n": 6144, "k": 2048},
        # The shared expert's gate and up of a ragged verify batch (sizes no tile divides), and
        # of a long prompt.
        {"name": "swiglu_int8_ragged", "op": "swiglu_int8", "m": 77, "n": 1360, "k": 1040},
        {"name": "swiglu_int8_long", "op": "swiglu_int8", "m": 4096, "n": 2048, "k": 6144},
        # Norm and shared expert together: a decode step's eight rows, a prefill sub-chunk.
        {"name": "mlp_int8_decode", "op": "mlp_int8", "rows": 8, "cols": 6144, "inter": 2048},
        {"name": "mlp_int8_chunk", "op": "mlp_int8", "rows": 256, "cols": 6144, "inter": 2048},
        # The routed layer of one token, and of eight decode rows, in the large configuration.
        {"name": "few_token", "op": "few", "rows": 1, "experts": 256, "top_k": 8, "cols": 6144,
         "inter": 2048, "shared": True},
        {"name": "few_decode", "op": "few", "rows": 8, "experts": 256, "top_k": 8, "cols": 6144,
         "inter": 2048, "shared": True},
        # Three drafted tokens verified on the small configuration, no shared expert.
        {"name": "few_small", "op": "few", "rows": 3, "experts": 64, "top_k": 8, "cols": 2048,
         "inter": 768, "shared": False},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "dense_int8", "swiglu_int8", "mlp_int8", "few"])
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 4096), "cols": _log_int(rng, 128, 6144, 16)}
    if op == "dense_int8":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 128, 6144, 16),
                "k": _log_int(rng, 128, 6144, 16)}
    if op == "swiglu_int8":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 128, 2048, 16),
                "k": _log_int(rng, 128, 6144, 16)}
    if op == "mlp_int8":
        return {"op": op, "rows": _log_int(rng, 1, 2048), "cols": _log_int(rng, 128, 6144, 16),
                "inter": _log_int(rng, 128, 2048, 16)}
    experts = _log_int(rng, 8, 256)
    top_k = min(rng.choice([1, 2, 4, 6, 8]), experts)
    rows = _log_int(rng, 1, 16)
    cols, inter = _log_int(rng, 512, 6144, 64), _log_int(rng, 128, 2048, 64)
    while rows * top_k * cols * inter > 64 * 6144 * 2048:
        cols = max(64, cols // 128 * 64)
    return {"op": op, "rows": rows, "experts": experts, "top_k": top_k, "cols": cols,
            "inter": inter, "shared": rng.random() < 0.5}


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------ inputs


def _hidden(gen, rows, cols):
    """BF16 hidden states: normal, one channel in 256 an outlier."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x[:, 5::256] *= 16.0
    return x.to(torch.bfloat16)


def _norm_weight(gen, cols):
    return (1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)


def _int8_rows(gen, rows, cols):
    """Quantised rows as the step before the product leaves them, and their scales."""
    x = _hidden(gen, rows, cols).float()
    scale = (x.abs().amax(1) / INT8_MAX).clamp(min=MIN_SCALE)
    return torch.round(x / scale[:, None]).to(torch.int8), scale


def _int8_weight(gen, n, k):
    """INT8 weight [n, k] of N(0, 1 / k) and one scale per output channel."""
    w = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
    scale = w.abs().amax(1) / INT8_MAX
    return torch.round(w / scale[:, None]).to(torch.int8), scale


def _nvfp4(gen, experts, n, k):
    """NVFP4 weights whose products with normal rows are of order one: packed codes, block
    scales (E4M3, one per 16 k) and one FP32 scale per expert."""
    packed = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, generator=gen,
                           device="cuda")
    scales = torch.empty((experts, n, k // 16), dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, min(experts, (1 << 27) // (n * (k // 16))))
    for e in range(0, experts, step):
        c = min(step, experts - e)
        v = torch.rand((c, n, k // 16), generator=gen, device="cuda") * 3.9375 + 0.0625
        scales[e:e + c] = v.to(torch.float8_e4m3fn)
    scale2 = (0.5 + 1.5 * torch.rand(experts, generator=gen, device="cuda")) / (7 * math.sqrt(k))
    return packed, scales, scale2


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    st = {"op": op}
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if op in ("norm", "mlp_int8"):
        rows, cols = case["rows"], case["cols"]
        st["x"] = _hidden(gen, rows, cols)
        st["res"] = (4.0 * torch.randn((rows, cols), generator=gen, device="cuda")).to(
            torch.bfloat16)
        st["g"] = _norm_weight(gen, cols)
        st["h"] = torch.empty((rows, cols), **bf)
    if op == "norm":
        st["y"] = torch.empty((rows, cols), **bf)
        st["q"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
        st["s"] = torch.empty((rows, _blocks(cols)), device="cuda")
    elif op == "mlp_int8":
        inter = case["inter"]
        st["gate"], st["up"] = _int8_weight(gen, inter, cols), _int8_weight(gen, inter, cols)
        st["down"] = _int8_weight(gen, cols, inter)
        st["q"] = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
        st["s"] = torch.empty(rows, device="cuda")
        if own:
            import grouped_nvfp4_w4a16_amd as hip

            st["mlp"] = hip.SharedExpertInt8(*st["gate"], *st["up"], *st["down"], rows)
    elif op in ("dense_int8", "swiglu_int8"):
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["sa"] = _int8_rows(gen, m, k)
        st["w"] = [_int8_weight(gen, n, k) for _ in range(2 if op == "swiglu_int8" else 1)]
        st["c"] = torch.empty((m, n), **bf)
    else:
        rows, experts, top_k = case["rows"], case["experts"], case["top_k"]
        cols, inter = case["cols"], case["inter"]
        st["x"] = torch.randn((rows, cols), generator=gen, device="cuda").to(torch.bfloat16)
        st["logits"] = torch.randn((rows, experts), generator=gen, device="cuda")
        st["top_k"] = top_k
        st["gate_up"] = _nvfp4(gen, experts, 2 * inter, cols)
        st["down"] = _nvfp4(gen, experts, cols, inter)
        st["shared"] = torch.randn((rows, cols), generator=gen, device="cuda").to(
            torch.bfloat16) if case["shared"] else None
        st["out"] = torch.empty((rows, cols), **bf)
        if own:
            import grouped_nvfp4_w4a16_amd as hip

            def table(w, n, k):
                return hip.ExpertTable(list(w[0].unbind(0)),
                                       list(w[1].view(torch.uint8).unbind(0)), w[2], n, k)

            st["gt"] = table(st["gate_up"], 2 * inter, cols)
            st["dt"] = table(st["down"], cols, inter)
            st["ws"] = hip.FewWorkspace(rows, top_k, inter)
    return st


# ------------------------------------------------------------------- the operators, plain


def _norm(st):
    """The stored sum h = x + residual (BF16, what the next layer adds to) and its norm, FP32."""
    h = (st["x"].float() + st["res"].float()).to(torch.bfloat16)
    f = h.float()
    return h, f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * st["g"].float()


def _quant_fp8(v):
    rows, cols = v.shape
    pad = torch.nn.functional.pad(v, (0, _blocks(cols) * BLOCK - cols))
    scale = (pad.view(rows, -1, BLOCK).abs().amax(2) / E4M3_MAX).clamp(min=MIN_SCALE)
    return (v / scale.repeat_interleave(BLOCK, 1)[:, :cols]).to(torch.float8_e4m3fn), scale


def _quant_int8(v):
    scale = (v.abs().amax(1) / INT8_MAX).clamp(min=MIN_SCALE)
    return torch.round(v / scale[:, None]), scale


def _product(a, sa, w):
    """INT8 codes (as FP32) times an INT8 weight, with the scales of token and channel."""
    return (a @ w[0].float().t()) * sa[:, None] * w[1]


def _swiglu(g, u):
    g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    return g / (1.0 + torch.exp(-g)) * u


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _slots(w, ids):
    """[slots, n, k] FP32 weights of each slot's expert (without the expert's scale)."""
    code = torch.tensor(_E2M1, device="cuda")
    pair = torch.stack((code.repeat(16), code.repeat_interleave(16)), 1)  # byte -> low, high
    v = pair[w[0][ids].int()]  # [slots, n, k / 2, 2]
    slots, n, half, _ = v.shape
    v = v.view(slots, n, half // 8, 16).mul_(w[1][ids].float()[..., None])
    return v.view(slots, n, 2 * half)


def _few(st):
    rows, top_k = st["x"].shape[0], st["top_k"]
    val, ids = st["logits"].topk(top_k, dim=1)  # softmax over the selected logits
    p = torch.exp(val - val[:, :1])
    p = p / p.sum(1, keepdim=True)
    ids = ids.view(-1)
    x = st["x"].float().repeat_interleave(top_k, 0)
    y = torch.bmm(_slots(st["gate_up"], ids), x[:, :, None])[:, :, 0]
    y = y * st["gate_up"][2][ids][:, None]
    inter = y.shape[1] // 2
    act = _swiglu(y[:, :inter], y[:, inter:])
    y = torch.bmm(_slots(st["down"], ids), act[:, :, None])[:, :, 0]
    y = y * (st["down"][2][ids] * p.view(-1))[:, None]
    y = y.view(rows, top_k, -1).sum(1)
    if st["shared"] is not None:
        y = y + st["shared"].float()
    return y.to(torch.bfloat16)


def _plain(st):
    op = st["op"]
    if op == "norm":
        h, y = _norm(st)
        return [h, y.to(torch.bfloat16), *_quant_fp8(y)]
    if op == "dense_int8":
        return [_product(st["a"].float(), st["sa"], st["w"][0]).to(torch.bfloat16)]
    if op == "swiglu_int8":
        a = st["a"].float()
        return [_swiglu(_product(a, st["sa"], st["w"][0]),
                        _product(a, st["sa"], st["w"][1])).to(torch.bfloat16)]
    if op == "mlp_int8":
        h, y = _norm(st)
        q, s = _quant_int8(y)
        act = _swiglu(_product(q, s, st["gate"]), _product(q, s, st["up"]))
        q, s = _quant_int8(act)
        return [h, _product(q, s, st["down"]).to(torch.bfloat16)]
    return [_few(st)]


def _hip(st):
    import grouped_nvfp4_w4a16_amd as hip

    op = st["op"]
    if op == "norm":
        hip.moe_rmsnorm_fp8(st["x"], st["g"], st["q"], st["s"], EPS, residual=st["res"],
                            h=st["h"], y=st["y"])
        return [st["h"], st["y"], st["q"], st["s"]]
    if op == "dense_int8":
        hip.moe_dense_gemm_int8(st["a"], st["sa"], *st["w"][0], st["c"])
        return [st["c"]]
    if op == "swiglu_int8":
        hip.moe_dense_gate_up_swiglu_int8(st["a"], st["sa"], *st["w"][0], *st["w"][1], st["c"],
                                          LIMIT)
        return [st["c"]]
    if op == "mlp_int8":
        hip.moe_rmsnorm_int8(st["x"], st["g"], st["q"], st["s"], EPS, residual=st["res"],
                             h=st["h"])
        return [st["h"], st["mlp"](st["q"], st["s"], LIMIT)]
    hip.moe_layer_few_from_logits(st["x"], st["logits"], st["top_k"], st["gt"], st["dt"], LIMIT,
                                  st["ws"], st["out"], shared=st["shared"])
    return [st["out"]]


def run(state):
    return _hip(state) if own else _plain(state)


# ------------------------------------------------------------------------- work and exact


def _experts_used(case):
    """How many experts the rows of such a case reach on average (uniform routing)."""
    miss = (1.0 - case["top_k"] / case["experts"]) ** case["rows"]
    return case["experts"] * (1.0 - miss)


def work(case):
    op = case["op"]
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        # x and residual in; h, y and the codes out; about ten operations per value
        return {"bytes": rows * (9 * cols + 4 * _blocks(cols)) + 2 * cols,
                "flops": 10 * rows * cols}
    if op in ("dense_int8", "swiglu_int8"):
        m, n, k = case["m"], case["n"], case["k"]
        n_w = 2 * n if op == "swiglu_int8" else n
        return {"bytes": n_w * (k + 4) + m * (k + 4) + 2 * m * n, "flops": 2 * m * n_w * k}
    if op == "mlp_int8":
        rows, cols, inter = case["rows"], case["cols"], case["inter"]
        return {"bytes": 3 * cols * inter + 4 * (2 * inter + cols) + 2 * cols + 8 * rows * cols,
                "flops": 6 * rows * cols * inter}
    rows, cols, inter = case["rows"], case["cols"], case["inter"]
    weights = 3 * cols * inter * 9 // 16  # codes and block scales of one expert
    return {"bytes": int(_experts_used(case) * weights) + 4 * rows * case["experts"] +
            (6 if case["shared"] else 4) * rows * cols,
            "flops": 6 * rows * case["top_k"] * cols * inter}


def _exact_norm(st):
    s = st["x"].double() + st["res"].double()
    h = s.to(torch.float32).to(torch.bfloat16)  # two BF16 numbers: FP32 between rounds nothing
    f = h.double()
    return s, f / torch.sqrt(f.pow(2).sum(1, keepdim=True) / f.shape[1] + EPS) * \
        st["g"].double()[None, :]


def _round_e4m3(v):
    """FP64 values to the nearest E4M3 value (ties to even), |v| <= 448 after rounding."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    ulp = torch.exp2(torch.clamp(e.double() - 1.0, min=-6.0) - 3.0)
    return torch.round(v / ulp) * ulp


def _exact_fp8(v):
    q, s = torch.empty_like(v), v.new_empty(v.shape[0], _blocks(v.shape[1]))
    for b in range(s.shape[1]):
        c = slice(b * BLOCK, min((b + 1) * BLOCK, v.shape[1]))
        s[:, b] = torch.clamp(v[:, c].abs().max(dim=1).values / E4M3_MAX, min=MIN_SCALE)
        q[:, c] = _round_e4m3(v[:, c] / s[:, b:b + 1])
    return [q, s]


def _exact_int8(v):
    s = torch.clamp(v.abs().max(dim=1).values / INT8_MAX, min=MIN_SCALE)
    return torch.round(v / s[:, None]), s


def _exact_product(a, sa, w):
    return torch.mm(a.double(), w[0].double().t()) * (sa.double()[:, None] *
                                                      w[1].double()[None, :])


def _exact_swiglu(g, u):
    g = torch.minimum(g, torch.full_like(g, LIMIT))
    u = torch.maximum(torch.minimum(u, torch.full_like(u, LIMIT)), torch.full_like(u, -LIMIT))
    return g * torch.sigmoid(g) * u


def _exact_weight(w, e):
    """Expert e's [n, k] weight in FP64: code value x block scale x expert scale."""
    code = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    b = w[0][e].long()
    v = torch.empty((b.shape[0], 2 * b.shape[1]), dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = code[b & 15], code[b >> 4]
    return v * w[1][e].double().repeat_interleave(16, 1) * w[2][e].double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        s, y = _exact_norm(st)
        return [s, y, *_exact_fp8(y)]
    if op == "dense_int8":
        return [_exact_product(st["a"], st["sa"], st["w"][0])]
    if op == "swiglu_int8":
        return [_exact_swiglu(*(_exact_product(st["a"], st["sa"], w) for w in st["w"]))]
    if op == "mlp_int8":
        s, y = _exact_norm(st)
        q = _exact_int8(y)
        act = _exact_swiglu(_exact_product(*q, st["gate"]), _exact_product(*q, st["up"]))
        return [s, _exact_product(*_exact_int8(act), st["down"])]
    logits = st["logits"].double().cpu().numpy()
    out = []
    for r in range(case["rows"]):
        ids = np.argsort(-logits[r], kind="stable")[:case["top_k"]]
        p = np.exp(logits[r, ids] - logits[r].max())
        p /= p.sum()
        x = st["x"][r].double()
        y = torch.zeros(case["cols"], dtype=torch.float64, device="cuda")
        for e, weight in zip(ids.tolist(), p.tolist()):
            gu = _exact_weight(st["gate_up"], e) @ x
            act = _exact_swiglu(gu[:case["inter"]], gu[case["inter"]:])
            y += weight * (_exact_weight(st["down"], e) @ act)
        out.append(y)
    y = torch.stack(out)
    return [y if st["shared"] is None else y + st["shared"].double()]

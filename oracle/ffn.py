"""The feed-forward half around the routed experts for the oracle (test infrastructure only), in
NumPy FP64: the residual's addition and the root-mean-square norm, INT8 rows and products, the
INT8 shared expert, and the routed NVFP4 layer of a few tokens.

- ``quantise_int8`` and ``int8_product`` are bit-exact: the operators define their FP32 steps.
- The others are the operators' formulas without any of their intermediate roundings, except the
  one each definition states (the stored sum of the norm).
"""

from __future__ import annotations

import numpy as np

from . import codecs, moe

INT8_MAX = np.float32(127.0)
MIN_SCALE = np.float32(2.0 ** -126)


def rmsnorm(x, weight, eps: float, residual=None):
    """(h, y): the sum rounded to BF16 (as FP64), and its norm, unrounded."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    h = codecs.round_bf16(s)
    mean = np.mean(h * h, axis=1, keepdims=True)
    return h, h / np.sqrt(mean + eps) * np.asarray(weight, np.float64)[None, :]


def quantise_int8(x):
    """(codes, scales) of FP32 rows, every step in FP32; a row that is not finite has codes 0."""
    x = np.asarray(x, np.float32)
    amax = np.max(np.abs(x), axis=1, initial=0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        s = (amax / INT8_MAX).astype(np.float32)
        s = np.where(s < MIN_SCALE, MIN_SCALE, s).astype(np.float32)
        q = np.rint((x / s[:, None]).astype(np.float32))
    q = np.where(np.isfinite(s)[:, None], q, 0.0)
    return q.astype(np.int8), s


def int8_values(a, a_scale, w, w_scale):
    """FP32 values ``(float(sum) * a_scale) * w_scale`` of the exact integer sums."""
    sums = np.asarray(a, np.float64) @ np.asarray(w, np.float64).T  # integers below 2^53: exact
    v = sums.astype(np.float32) * np.asarray(a_scale, np.float32)[:, None]
    return (v * np.asarray(w_scale, np.float32)[None, :]).astype(np.float32)


def int8_product(a, a_scale, w, w_scale):
    """The BF16 output of the dense product, as FP64."""
    return codecs.round_bf16(int8_values(a, a_scale, w, w_scale).astype(np.float64))


def int8_swiglu(a, a_scale, gate, gate_scale, up, up_scale, limit: float):
    """silu(min(G, L)) clamp(U, -L, L) of the FP32 values, unrounded."""
    g = int8_values(a, a_scale, gate, gate_scale).astype(np.float64)
    u = int8_values(a, a_scale, up, up_scale).astype(np.float64)
    return moe.swiglu_clamp(g, u, limit)


def code_values(packed, scales):
    """NVFP4 weights without their expert's scale: E2M1 value times E4M3 block scale."""
    return moe.dequant(packed, scales, 1.0, "exact")


def few_layer(x, topk_ids, topk_weights, gate_up, down, scale2_gate_up, scale2_down, limit: float,
              shared=None):
    """``(out, bound_terms)`` of the routed layer; an expert is a ``(packed, scales)`` pair or None.

    ``bound_terms`` holds, per covered slot, what error bounds need: the row, the weight, and the
    gate, up and activation values with the sums of their products' magnitudes."""
    x = np.asarray(x, np.float64)
    ids = np.asarray(topk_ids, np.int64)
    rows, top_k = ids.shape
    n_exp = len(gate_up)
    hidden = x.shape[1]
    out = np.zeros((rows, hidden))
    terms = []
    for r in range(rows):
        seen = set()
        for j in range(top_k):
            e = int(ids[r, j])
            if not 0 <= e < n_exp or e in seen or gate_up[e] is None or down[e] is None:
                continue
            seen.add(e)
            w1, w2 = code_values(*gate_up[e]), code_values(*down[e])
            s1, s2 = float(np.float32(scale2_gate_up[e])), float(np.float32(scale2_down[e]))
            gu = (w1 @ x[r]) * s1
            mi = gu.size // 2
            act = moe.swiglu_clamp(gu[None, :mi], gu[None, mi:], limit)[0]
            p = float(np.float32(topk_weights[r, j]))
            out[r] += p * s2 * (w2 @ act)
            terms.append(dict(row=r, p=p * s2, gate=gu[:mi], up=gu[mi:], act=act, down=w2,
                              mag=(np.abs(w1) @ np.abs(x[r])) * abs(s1)))
    if shared is not None:
        out = out + np.asarray(shared, np.float64)
    return out, terms

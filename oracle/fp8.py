"""FP8 (E4M3, one FP32 scale per block of 128) definitions for the oracle (test
infrastructure only): quantisation of rows, the block-scaled product, the grouped product and
the routed layer, in NumPy FP64.

- ``quantise_rows`` is bit-exact for FP32 inputs: the two divisions are IEEE FP32 ones
  (NumPy's), as the definition of the operator states, and the rounding to E4M3 is exact.
- Products are FP64 sums of exact products; only the outputs the operators store are rounded
  (by the caller, where a test wants it).
"""

from __future__ import annotations

import numpy as np

from . import codecs, moe

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = np.float32(2.0 ** -126)


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def round_e4m3(v):
    """FP64 values to the nearest E4M3 value, ties to even. Magnitudes that would round past
    448 (past 464) have no E4M3 value: NaN, like a NaN input."""
    v = np.asarray(v, dtype=np.float64)
    _, exp = np.frexp(v)  # |v| in [2^(exp-1), 2^exp)
    quantum = np.maximum(exp - 1, -6) - 3  # 3 mantissa bits; subnormals below 2^-6
    with np.errstate(invalid="ignore"):
        r = np.ldexp(np.rint(np.ldexp(v, -quantum)), quantum)
        return np.where(np.abs(r) <= E4M3_MAX, r, np.nan)


def e4m3_codes(v):
    """Codes (uint8) of FP64 values that are E4M3 values; NaN gives 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    table = codecs.e4m3fn_decode(np.arange(0x7F))  # the non-negative finite codes, increasing
    mag = np.searchsorted(table, np.abs(np.nan_to_num(v)))
    mag = np.where(np.isnan(v), 0x7F, mag)
    return (mag | np.where(np.signbit(v) & ~np.isnan(v), 0x80, 0)).astype(np.uint8)


def scales_of(x):
    """FP32 scale per row and block of FP32 (or FP64) values [rows, cols]: max(amax / 448,
    2^-126), NaN where the block holds one."""
    x = np.asarray(x)
    rows, cols = x.shape
    out = np.empty((rows, blocks(cols)), np.float32)
    for b in range(out.shape[1]):
        amax = np.max(np.abs(x[:, b * BLOCK:(b + 1) * BLOCK]), axis=1).astype(np.float32)
        s = amax / np.float32(E4M3_MAX)
        out[:, b] = np.where(s < MIN_SCALE, MIN_SCALE, s)
    return out


def expand(scale, cols: int):
    """Row scales [rows, blocks] as one value per column."""
    return np.repeat(np.asarray(scale), BLOCK, axis=1)[:, :cols]


def quantise_rows(x):
    """(values, scale) of FP32 rows: values are E4M3 values in FP64 (NaN possible)."""
    x = np.asarray(x, dtype=np.float32)
    s = scales_of(x)
    with np.errstate(invalid="ignore", over="ignore"):
        q = x / expand(s, x.shape[1])  # FP32
    return round_e4m3(q.astype(np.float64)), s


def weight(codes, scale):
    """FP64 weight [n, k] of E4M3 codes and FP32 block scales [n / 128, k / 128]."""
    n, k = np.shape(codes)
    s = np.repeat(np.asarray(scale, np.float64), BLOCK, axis=0)[:n]
    return codecs.e4m3fn_decode(codes) * expand(s, k)


def rows_f64(codes, scale):
    return codecs.e4m3fn_decode(codes) * expand(np.asarray(scale, np.float64), np.shape(codes)[1])


def product(a_codes, a_scale, w_codes, w_scale):
    """[m, n] FP64 products of the values the codes and scales stand for."""
    return rows_f64(a_codes, a_scale) @ weight(w_codes, w_scale).T


def swiglu_product(a_codes, a_scale, gate, up, limit: float):
    """silu(min(G, L)) * clamp(U, -L, L) in FP64; ``gate`` and ``up`` are (codes, scale)."""
    return moe.swiglu_clamp(product(a_codes, a_scale, *gate), product(a_codes, a_scale, *up),
                            limit)


def split_gate_up(codes, scale):
    """The (gate, up) halves of a fused gate_up weight and its scales."""
    mi, nb = np.shape(codes)[0] // 2, np.shape(scale)[0] // 2
    return (codes[:mi], scale[:nb]), (codes[mi:], scale[nb:])


def segments(expert_offsets, max_rows: int):
    """(expert, first row, end row) of every expert with rows."""
    for e in range(len(expert_offsets) - 1):
        lo, hi = max(int(expert_offsets[e]), 0), min(int(expert_offsets[e + 1]), max_rows)
        if lo < hi:
            yield e, lo, hi


def gathered(a_codes, a_scale, index):
    """Rows of (codes, scale) at ``index``; an index out of range gives zeros."""
    index = np.asarray(index)
    ok = (index >= 0) & (index < len(a_codes))
    safe = np.where(ok, index, 0)
    return (np.where(ok[:, None], np.asarray(a_codes)[safe], 0).astype(np.uint8),
            np.where(ok[:, None], np.asarray(a_scale)[safe], 0).astype(np.float32))


def moe_layer(x, topk_ids, topk_weights, gate_up, down, limit: float, shared=None):
    """The routed FP8 layer in FP64 from FP32 rows ``x``: x quantised, per expert the SwiGLU
    product, its output quantised from its FP32 rounding, the down product rounded to BF16,
    the top-k sum (not rounded). ``gate_up`` and ``down`` hold (codes, scale) or None."""
    v, s = quantise_rows(x)
    xq = e4m3_codes(v)
    out = np.zeros((x.shape[0], x.shape[1]))
    for r in range(x.shape[0]):
        for j in range(topk_ids.shape[1]):
            e = int(topk_ids[r, j])
            if not 0 <= e < len(gate_up) or gate_up[e] is None:
                continue
            g, u = split_gate_up(*gate_up[e])
            act = swiglu_product(xq[r:r + 1], s[r:r + 1], g, u, limit)
            av, as_ = quantise_rows(act.astype(np.float32))
            y = product(e4m3_codes(av), as_, *down[e])
            out[r] += float(topk_weights[r, j]) * codecs.round_bf16(y)[0]
    if shared is not None:
        out += shared
    return out

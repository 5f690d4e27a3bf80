"""Inputs of the few-token layer whose gate and up sums are exact, and tight error bounds for them.

Rows of -1, 0 and 1 against weights of ``workloads.random_nvfp4``: every product is a multiple of 2^-8
(E2M1 values of multiples of 0.5, block scales of at least 2^-4 with 4 significant bits), so FP32 sums
are exact in any order while the magnitudes add up to less than 2^16 (``assert_exact``). Gate and up
then carry one rounding, that of scale2. u = 2^-24. silu's slope is at most 1.1. The SwiGLU's own
error is (|g| + 8) u <= 2^-17. Activations stay below B = limit max(limit, 0.2785) (silu's least value
is -0.27846...); limits up to 128 store them in FP16 times a power of two that brings B to [2^14,
2^15): off by 2^-11 of themselves or by half of FP16's smallest step there, 2^-25 2^-14 B. The down
products are exact in FP32, a sum of mi of them is off by (mi + 64) u of their magnitudes, and the
BF16 output by 2^-8 of itself."""

import numpy as np

from oracle import ffn

U = 2.0 ** -24


def signs(rng, rows, hidden):
    """BF16 bits of rows of -1, 0 (one in eight) and 1."""
    v = rng.choice([-1.0, 1.0], (rows, hidden)) * (rng.random((rows, hidden)) >= 0.125)
    return (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def assert_exact(gate_up, rows, step=1.0):
    """The magnitudes of every sum of these rows (FP64, multiples of `step`) stay below 2^16 step."""
    assert np.array_equal(np.rint(rows / step) * step, rows)
    most = np.abs(rows).max(axis=0)
    for w in gate_up:
        assert w is None or (np.abs(ffn.code_values(*w)) @ most).max() < 2.0 ** 16 * step


def bounds(ref, terms, limit):
    """Per element bounds of a layer (``ffn.few_layer``'s results) with exact gate and up sums."""
    assert limit <= 128
    elem = np.abs(ref) * 2.0 ** -8 + 2.0 ** -130
    store = limit * max(limit, 0.2785) * 2.0 ** -39
    for t in terms:
        mi = t["act"].size
        u_c = np.abs(np.clip(t["up"], -limit, limit))
        act = np.abs(t["act"])
        d_act = 1.1 * np.abs(t["gate"]) * U * u_c + act * (U + 2.0 ** -11 + 2.0 ** -17) + store
        elem[t["row"]] += abs(t["p"]) * (np.abs(t["down"]) @ (d_act + (mi + 64) * U * act))
    return elem

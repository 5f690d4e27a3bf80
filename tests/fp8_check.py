"""Bounds and checks for the SwiGLU products' quantised outputs (test infrastructure only).

v = silu(min(G, L)) * clamp(U, -L, L) is known in FP64; a kernel computes it in FP32 and writes
codes and a scale per 128 columns. ``Expected`` bounds the FP32 value's error element by element,
and ``check`` holds scales and codes to what that allows, so that a code may only differ where
the value lies as close to a border of two codes as the bound."""

import copy

import numpy as np

from oracle import codecs, fp8

BASE = 3.0  # standard deviation of the gate and up sums: below the limit of 7, mostly


def exact_operand(rng, rows, k, block_rows):
    """Codes of {-2, .., 2}, power-of-two scales: products are whole multiples (at most 64) of a
    common quantum, so that a sum of up to 2^18 of them is exact in FP32 in every order. A
    product's deviation is 2 * 1.75, which the scales bring to about BASE for a sum of k."""
    vals = rng.integers(-2, 3, (rows, k)).astype(np.float64)
    n_s = fp8.blocks(rows) if block_rows else rows
    scale = np.exp2(rng.integers(-1, 2, (n_s, fp8.blocks(k))))
    if block_rows:
        scale *= np.exp2(np.round(np.log2(BASE / (3.5 * np.sqrt(k)))))
    return fp8.e4m3_codes(vals), scale.astype(np.float32)


def normal_operand(rng, rows, k, block_rows):
    """Rows quantised from N(0, 1); weights' codes of the same kind with block scales that
    bring a sum of k to about BASE (a code's deviation is 448 over the largest of 128: 160)."""
    v = rng.standard_normal((rows, k)).astype(np.float32)
    q, s = fp8.quantise_rows(v)
    if block_rows:
        s = rng.uniform(0.5, 1.5, (fp8.blocks(rows), fp8.blocks(k))) * BASE / np.sqrt(k) / 160
    return fp8.e4m3_codes(q), s.astype(np.float32)


def sum_error(a, sa, w, sw):
    """Bound on |FP32 sum - exact|: a term passes at most 128 additions inside its block of k,
    the rounding of the two scales' product, an FMA per block and the joins of at most 8
    splits; each moves it by at most a step (2^-23, rounded or cut) of a partial sum, which
    the sum of magnitudes bounds."""
    total = np.abs(fp8.rows_f64(a, sa)) @ np.abs(fp8.weight(w, sw)).T
    return (128 + 1 + fp8.blocks(a.shape[1]) + 8) * 2.0 ** -23 * 1.001 * total


class Expected:
    """v of a row block's gate and up sums (FP64) and the bound ``err`` on |FP32 value - v|."""

    def __init__(self, g, u, g_err, u_err, limit):
        gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit)
        silu = gc / (1 + np.exp(-gc))
        self.v = silu * uc
        # |silu'| <= 1.1, the clamps change no more than their argument; then e^-|g| (|g| times
        # the rounding of its exponent), its and the reciprocal's ulp, one sum, three products
        self.err = 1.1 * g_err * (np.abs(uc) + u_err) + np.abs(silu) * u_err + \
            np.abs(self.v) * (2.25 * np.abs(gc) + 10) * 2.0 ** -24 + 2.0 ** -140
        self.plain = float(np.mean((g < limit) & (np.abs(u) < limit)))

    def rows(self, index):
        """The same for these rows."""
        part = copy.copy(self)
        part.v, part.err = self.v[index], self.err[index]
        return part


def expected(a, sa, gate, up, limit, exact):
    zero = 0.0
    g, u = fp8.product(a, sa, *gate), fp8.product(a, sa, *up)
    return Expected(g, u, zero if exact else sum_error(a, sa, *gate),
                    zero if exact else sum_error(a, sa, *up), limit)


def check(codes, scale, want):
    """Raises unless the codes and scales are those of FP32 values within ``want``'s bounds."""
    rows, cols = want.v.shape
    assert codes.shape == (rows, cols) and scale.shape == (rows, fp8.blocks(cols))
    step = 2.0 ** -23  # of a division: twice its rounding
    for b in range(fp8.blocks(cols)):
        c = slice(b * fp8.BLOCK, min((b + 1) * fp8.BLOCK, cols))
        v, err = want.v[:, c], want.err[:, c]
        mag = np.abs(v)
        # the test has to be able to tell: bounds far below the group's largest value
        assert np.all(np.max(err, axis=1) <= 2.0 ** -6 * np.maximum(np.max(mag, axis=1), 2.0 ** -120))
        s = scale[:, b].astype(np.float64)
        lo = np.maximum(np.max(mag - err, axis=1) / 448 * (1 - step), 2.0 ** -126)
        hi = np.maximum(np.max(mag + err, axis=1) / 448 * (1 + step), 2.0 ** -126)
        assert np.all((s >= lo) & (s <= hi)), ("scale", b, float(np.max(np.abs(s / lo - 1))))
        s = s[:, None]
        q0, q1 = (v - err) / s, (v + err) / s
        q0, q1 = q0 - step * np.abs(q0), q1 + step * np.abs(q1)
        got = codecs.e4m3fn_decode(codes[:, c])
        ok = (got >= fp8.round_e4m3(np.clip(q0, -448, 448))) & \
            (got <= fp8.round_e4m3(np.clip(q1, -448, 448)))
        assert np.all(ok), ("codes", b, int(np.sum(~ok)))

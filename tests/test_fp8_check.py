"""The checks of the SwiGLU products' outputs accept the operator's FP32 form and reject wrong
ones: without a GPU, on results planted in the reference."""

import functools

import numpy as np
import pytest

import fp8_check
from oracle import fp8

LIMIT = 7.0


def _fp32(g, u, limit=LIMIT):
    """The operator in FP32 from FP64 sums rounded to FP32."""
    g, u = g.astype(np.float32), u.astype(np.float32)
    gc, uc = np.minimum(g, np.float32(limit)), np.clip(u, np.float32(-limit), np.float32(limit))
    v = (gc / (np.float32(1) + np.exp(-gc)) * uc).astype(np.float32)
    q, s = fp8.quantise_rows(v)
    return fp8.e4m3_codes(q), s


def _roll(scale, axis):
    return np.roll(scale, 1, axis=axis)


WRONG = {
    "zeros": lambda g, u, part: (0 * g, u),
    "sign": lambda g, u, part: (g, -u),
    "gate and up exchanged": lambda g, u, part: (u, g),
    "last block of k dropped": lambda g, u, part: part("drop"),
    "first block of k twice": lambda g, u, part: part("twice"),
    "row scales a block of k on": lambda g, u, part: part("roll rows"),
    "weight scales a block of k on": lambda g, u, part: part("roll weights"),
    "sums 1 % off": lambda g, u, part: (g * 1.01, u * 1.01),
    "rows moved by one": lambda g, u, part: (np.roll(g, 1, 0), np.roll(u, 1, 0)),
    "columns moved by four": lambda g, u, part: (np.roll(g, 4, 1), np.roll(u, 4, 1)),
}
SIZES = [(1, 144, 6144), (5, 272, 656), (40, 144, 2064)]


@functools.lru_cache(None)
def _operands(m, n, k, exact):
    rng = np.random.default_rng(m + n + k)
    make = fp8_check.exact_operand if exact else fp8_check.normal_operand
    return make(rng, m, k, False), make(rng, n, k, True), make(rng, n, k, True)


def _sums(rows, gate, up):
    return fp8.product(*rows, *gate), fp8.product(*rows, *up)


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_accepts_the_operator(m, n, k, exact):
    rows, gate, up = _operands(m, n, k, exact)
    want = fp8_check.expected(*rows, gate, up, LIMIT, exact)
    assert want.plain > 0.8  # gate and up within the limit: neither clamp hides the sums
    fp8_check.check(*_fp32(*_sums(rows, gate, up)), want)


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("name", WRONG)
def test_rejects(m, n, k, exact, name):
    if m == 1 and name == "rows moved by one":
        pytest.skip("one row")
    rows, gate, up = _operands(m, n, k, exact)
    want = fp8_check.expected(*rows, gate, up, LIMIT, exact)

    def part(kind):
        a, sa = rows
        last = (fp8.blocks(k) - 1) * fp8.BLOCK
        if kind == "drop":
            a = a.copy()
            a[:, last:] = 0
        if kind == "twice":
            first = fp8.product(a[:, :128], sa[:, :1], gate[0][:, :128], gate[1][:, :1])
            g, u = _sums(rows, gate, up)
            return g + first, u
        if kind == "roll rows":
            sa = _roll(sa, 1)
        if kind == "roll weights":
            return _sums((a, sa), (gate[0], _roll(gate[1], 1)), (up[0], _roll(up[1], 1)))
        return _sums((a, sa), gate, up)

    with pytest.raises(AssertionError):
        fp8_check.check(*_fp32(*WRONG[name](*_sums(rows, gate, up), part)), want)


def test_rejects_values_that_are_not_clamped():
    rows, gate, up = _operands(40, 144, 2064, True)
    want = fp8_check.expected(*rows, gate, up, LIMIT, True)
    with pytest.raises(AssertionError):
        fp8_check.check(*_fp32(*_sums(rows, gate, up), limit=100.0), want)


def test_rejects_sums_of_fewer_bits():
    """Exact sums pin the scales to FP32: 2.4e-5 off is too much (what the FP8 matrix cores'
    sums left in them)."""
    rows, gate, up = _operands(5, 272, 656, True)
    want = fp8_check.expected(*rows, gate, up, LIMIT, True)
    g, u = _sums(rows, gate, up)
    codes, scale = _fp32(g, u)
    with pytest.raises(AssertionError):
        fp8_check.check(codes, (scale * np.float32(1 + 2.4e-5)).astype(np.float32), want)
    with pytest.raises(AssertionError):
        fp8_check.check(codes, scale * np.float32(np.nan), want)

"""Pins of oracle/ffn.py against closed forms, exact rationals and torch."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import codecs, ffn, moe


def test_rmsnorm_of_constant_rows_is_the_weight():
    x = np.full((3, 8), 2.0)
    g = np.arange(8) / 4
    h, y = ffn.rmsnorm(x, g, 0.0)
    assert np.array_equal(h, x) and np.allclose(y, np.tile(g, (3, 1)), rtol=1e-15)


def test_rmsnorm_against_torch():
    rng = np.random.default_rng(1)
    x, r = (codecs.round_bf16(rng.standard_normal((5, 96))) for _ in range(2))
    g = codecs.round_bf16(rng.standard_normal(96))
    h, y = ffn.rmsnorm(x, g, 1e-3, r)
    t = (torch.tensor(x).bfloat16() + torch.tensor(r).bfloat16()).double()
    assert np.array_equal(h, t.numpy())
    want = torch.nn.functional.rms_norm(t, (96,), torch.tensor(g), 1e-3)
    assert np.allclose(y, want.numpy(), rtol=1e-13)


def test_int8_codes_by_exact_rationals():
    rng = np.random.default_rng(2)
    x = codecs.round_bf16(rng.standard_normal((4, 40)) * np.array([[1], [1e-30], [300], [0]]))
    q, s = ffn.quantise_int8(x)
    assert q.min() >= -127 and q.max() <= 127
    assert s[3] == np.float32(2.0 ** -126) and not q[3].any()
    for r in range(3):
        assert abs(int(q[r, np.argmax(np.abs(x[r]))])) == 127
        for c in range(40):
            quotient = np.float32(x[r, c]) / s[r]  # IEEE
            f = Fraction(float(quotient))
            assert abs(f - int(q[r, c])) <= Fraction(1, 2)
            if abs(f - int(q[r, c])) == Fraction(1, 2):
                assert int(q[r, c]) % 2 == 0


def test_int8_rows_that_are_not_finite():
    q, s = ffn.quantise_int8(np.array([[1.0, np.nan, 2.0], [np.inf, 1.0, -np.inf]]))
    assert np.isnan(s[0]) and np.isinf(s[1]) and not q.any()


def test_int8_product_one_hot_and_extremes():
    a = np.eye(16, dtype=np.int8)[:5] * 100
    w = np.arange(-128, 128, dtype=np.int16).astype(np.int8).reshape(16, 16)
    one = np.ones(16, np.float32)
    got = ffn.int8_product(a, one[:5], w, one)
    assert np.array_equal(got, codecs.round_bf16(100.0 * w[:, :5].T.astype(np.float64)))
    k = 131056  # the longest sums stay exact
    a, w = np.full((1, k), -128, np.int8), np.full((1, k), -128, np.int8)
    assert ffn.int8_values(a, one[:1], w, one[:1])[0, 0] == np.float32(128 * 128 * k)


def test_few_layer_against_the_sorted_oracle():
    """With power-of-two expert scales the BF16-weight oracle's weights are the exact products."""
    rng = np.random.default_rng(3)
    e, h, mi = 5, 256, 256
    gu = [wl.random_nvfp4(rng, 2 * mi, h) for _ in range(e)]
    dn = [wl.random_nvfp4(rng, h, mi) for _ in range(e)]
    gu[3] = dn[3] = None
    s1, s2 = np.full(e, 2.0 ** -7, np.float32), np.full(e, 0.25, np.float32)
    x = codecs.round_bf16(rng.standard_normal((3, h)))
    ids = np.array([[0, 4], [3, 1], [-1, 0]], np.int32)
    w = rng.random((3, 2)).astype(np.float32)
    got, terms = ffn.few_layer(x, ids, w, gu, dn, s1, s2, 7.0)
    want, _ = moe.moe_layer(x, ids, w, gu, dn, s1, s2, mi, 7.0, "exact")
    assert len(terms) == 4
    assert np.allclose(got, want, rtol=0, atol=0.02 * np.abs(want).max())  # its BF16 buffers
    # a repeated expert counts once, as a slot of its own row
    got2, _ = ffn.few_layer(x, np.array([[0, 0], [3, 1], [-1, 0]], np.int32), w, gu, dn, s1, s2, 7.0)
    once, _ = ffn.few_layer(x, np.array([[0, -1], [3, 1], [-1, 0]], np.int32), w, gu, dn, s1, s2, 7.0)
    assert np.array_equal(got2, once)


@pytest.mark.parametrize("rows", [0, 2])
def test_few_layer_without_experts_is_the_shared_term(rows):
    x = np.ones((rows, 64))
    out, terms = ffn.few_layer(x, np.full((rows, 2), -1), np.ones((rows, 2), np.float32), [None],
                               [None], [1.0], [1.0], 7.0, shared=3 * x)
    assert np.array_equal(out, 3 * x) and terms == []

"""The FP8 oracle (oracle/fp8.py) against torch's E4M3 conversion, exact rationals and closed
forms."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import codecs, fp8


def _torch_e4m3(v32):
    return torch.from_numpy(np.ascontiguousarray(v32)).to(torch.float8_e4m3fn)


def test_round_e4m3_against_torch_at_values_midpoints_and_neighbours():
    vals = codecs.e4m3fn_decode(np.arange(0x7F))
    mids = (vals[1:] + vals[:-1]) / 2
    base = np.concatenate([vals, mids, [448.0, 455.0, 463.9]]).astype(np.float32)
    near = np.concatenate([base, np.nextafter(base, np.float32(1e9)),
                           np.nextafter(base, np.float32(-1e9))])
    near = near[np.abs(near) < 464]
    near = np.concatenate([near, -near])
    got = fp8.round_e4m3(near.astype(np.float64))
    want = _torch_e4m3(near).double().numpy()
    assert np.array_equal(got, want)
    assert fp8.round_e4m3([464.0])[0] == 448.0  # a tie, to the even 448
    assert np.all(np.isnan(fp8.round_e4m3([464.1, 1e5, np.inf, np.nan])))


def test_round_e4m3_against_torch_on_random_values():
    rng = np.random.default_rng(3)
    v = (rng.standard_normal(200000) * np.exp2(rng.uniform(-14, 8, 200000))).astype(np.float32)
    v = v[np.abs(v) < 460]
    assert np.array_equal(fp8.round_e4m3(v.astype(np.float64)), _torch_e4m3(v).double().numpy())


def test_codes_round_trip():
    codes = np.arange(256).astype(np.uint8)
    finite = codes[(codes & 0x7F) != 0x7F]
    assert np.array_equal(fp8.e4m3_codes(codecs.e4m3fn_decode(finite)), finite)
    assert fp8.e4m3_codes([np.nan])[0] == 0x7F


def test_scales_closed_forms():
    x = np.zeros((4, 272), np.float32)
    x[0, 5] = -448.0
    x[1, 130] = 1.0
    x[2, 271] = 2.0 ** -140
    x[3, 0] = np.inf
    s = fp8.scales_of(x)
    assert s.shape == (4, 3) and s.dtype == np.float32
    assert s[0, 0] == 1.0 and s[1, 1] == np.float32(1) / np.float32(448)
    assert s[2, 2] == np.float32(2.0 ** -126) and s[0, 1] == np.float32(2.0 ** -126)
    assert np.isinf(s[3, 0])
    x[3, 1] = np.nan
    assert np.isnan(fp8.scales_of(x)[3, 0])


def test_quantised_values_are_within_half_a_step_and_never_saturate():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((64, 400)) * np.exp2(rng.uniform(-30, 30, (64, 1)))).astype(np.float32)
    q, s = fp8.quantise_rows(x)
    assert np.all(np.isfinite(q)) and np.max(np.abs(q)) <= 448
    back = q * fp8.expand(s.astype(np.float64), 400)
    # half a step: 2^-4 of the value, or half of 2^-9 scales below the normal range
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x) * (1 + 2.0 ** -20),
                                                 2.0 ** -10 * fp8.expand(s, 400) * 1.0001))


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (3, 144, 272)])
def test_product_against_exact_rationals(m, n, k):
    rng = np.random.default_rng(5)
    a = rng.integers(0, 0x7F, (m, k)).astype(np.uint8) | (rng.integers(0, 2, (m, k)) << 7).astype(np.uint8)
    w = rng.integers(0, 0x7F, (n, k)).astype(np.uint8)
    sa = np.exp2(rng.integers(-3, 3, (m, fp8.blocks(k)))).astype(np.float32)
    sw = rng.uniform(0.5, 2, (fp8.blocks(n), fp8.blocks(k))).astype(np.float32)
    got = fp8.product(a, sa, w, sw)
    dec = codecs.e4m3fn_decode(np.arange(256))
    for i, j in [(0, 0), (m - 1, n - 1), (m // 2, n // 2)]:
        want = Fraction(0)
        for q in range(k):
            want += (Fraction(dec[a[i, q]]) * Fraction(dec[w[j, q]]) *
                     Fraction(float(sa[i, q // 128])) * Fraction(float(sw[j // 128, q // 128])))
        mag = max(abs(float(want)), 1.0)
        assert abs(got[i, j] - float(want)) <= 1e-12 * mag * k


def test_layer_reduces_to_one_expert_by_hand():
    rng = np.random.default_rng(6)
    h, mi = 32, 16
    x = rng.standard_normal((2, h)).astype(np.float32)
    gu = (rng.integers(0, 0x40, (2 * mi, h)).astype(np.uint8), np.full((2, 1), 0.01, np.float32))
    dn = (rng.integers(0, 0x40, (h, mi)).astype(np.uint8), np.full((1, 1), 0.02, np.float32))
    ids = np.array([[0, 1], [1, -1]], np.int32)  # expert 1 absent
    wts = np.array([[0.75, 0.25], [1.0, 0.5]], np.float32)
    out = fp8.moe_layer(x, ids, wts, [gu, None], [dn, None], 7.0)
    v, s = fp8.quantise_rows(x[:1])
    xr = v * s.astype(np.float64)
    g = xr @ (codecs.e4m3fn_decode(gu[0][:mi]) * np.float64(np.float32(0.01))).T
    u = xr @ (codecs.e4m3fn_decode(gu[0][mi:]) * np.float64(np.float32(0.01))).T
    gc = np.minimum(g, 7.0)
    act = gc / (1 + np.exp(-gc)) * np.clip(u, -7, 7)
    av, as_ = fp8.quantise_rows(act.astype(np.float32))
    y = (av * as_.astype(np.float64)) @ (codecs.e4m3fn_decode(dn[0]) * np.float64(np.float32(0.02))).T
    assert np.allclose(out[0], 0.75 * codecs.round_bf16(y[0]), rtol=1e-12)
    assert np.all(out[1] == 0)

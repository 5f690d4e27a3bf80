"""moe_rmsnorm_bf16, moe_rmsnorm_fp8, moe_rmsnorm_int8 and moe_quant_int8 against the FP64 oracle.

Bounds. The stored sum is exact (two BF16 numbers' FP32 sum rounds to BF16 as the exact one does).
The norm's FP32 chain: at most cols / 1024 + 40 additions on a path of the sum (halved by the
root), and 8 roundings after it: relative error below ((cols / 2048 + 20) + 8) 2^-24 = CHAIN. A BF16
output adds 2^-8 of the value, a code half a step of its format at the value (E4M3: 2^-4 of it,
at least 2^-10 scales; INT8: half a scale), and the scale itself CHAIN + one division's rounding.
"""

import numpy as np
import pytest
import torch

import workloads as wl
from gpu_util import bf16_bits_host, bf16_dev, f64
from oracle import codecs, ffn, fp8

pytestmark = pytest.mark.gpu
BF16, F8, I8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8
TINY = 2.0 ** -125


def chain(cols):
    return (cols / 2048 + 28) * 2.0 ** -24


def _inputs(rows, cols, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * scale
    x[:, 3::97] *= 16
    r = rng.standard_normal((rows, cols)) * 4 * scale
    g = 1 + 0.2 * rng.standard_normal(cols)
    return [wl._to_bf16_bits(v.astype(np.float32)) for v in (x, r, g)]


def _values(bits):
    return codecs.bf16_bits_to_f64(bits)


# one lane, partial groups, one iteration, several, registers' limits, the loop past them
SIZES = [(1, 8), (3, 24), (5, 128), (2, 136), (7, 2048), (4, 6144), (3, 8200), (2, 32768),
         (2, 32776), (1, 70000), (600, 264), (513, 6144)]


def _check_y(got, want, cols):
    bound = np.abs(want) * (2.0 ** -8 + 2 * chain(cols)) + TINY
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_in_every_form(hip, rows, cols, residual):
    xb, rb, gb = _inputs(rows, cols, rows * 131 + cols)
    h_ref, y_ref = ffn.rmsnorm(_values(xb), _values(gb), 1e-5, _values(rb) if residual else None)
    x, r, g = bf16_dev(xb), bf16_dev(rb) if residual else None, bf16_dev(gb)
    h, y = torch.empty_like(x), torch.empty_like(x)
    hip.moe_rmsnorm_bf16(x, g, y, 1e-5, residual=r, h=h)
    assert np.array_equal(f64(h), h_ref)
    _check_y(f64(y), y_ref, cols)
    y_bits = bf16_bits_host(y)

    q, s = torch.empty((rows, cols), dtype=F8, device="cuda"), torch.empty(
        (rows, -(-cols // 128)), device="cuda")
    h2, y2 = torch.empty_like(x), torch.empty_like(x)
    hip.moe_rmsnorm_fp8(x, g, q, s, 1e-5, residual=r, h=h2, y=y2)
    assert np.array_equal(f64(h2), h_ref) and np.array_equal(bf16_bits_host(y2), y_bits)
    s_ref = fp8.scales_of(y_ref).astype(np.float64)
    assert np.all(np.abs(f64(s) - s_ref) <= s_ref * (2 * chain(cols) + 2.0 ** -22))
    se = fp8.expand(s_ref, cols)
    step = np.maximum(np.abs(y_ref) * 2.0 ** -4, se * 2.0 ** -10)
    err = np.abs(f64(q) * fp8.expand(f64(s), cols) - y_ref)
    assert np.all(err <= step * (1 + 2.0 ** -10) + np.abs(y_ref) * 8 * chain(cols))

    q8, s8 = torch.empty((rows, cols), dtype=I8, device="cuda"), torch.empty(rows, device="cuda")
    h3, y3 = torch.empty_like(x), torch.empty_like(x)
    hip.moe_rmsnorm_int8(x, g, q8, s8, 1e-5, residual=r, h=h3, y=y3)
    assert np.array_equal(f64(h3), h_ref) and np.array_equal(bf16_bits_host(y3), y_bits)
    s_ref = np.maximum(np.max(np.abs(y_ref), axis=1) / 127, 2.0 ** -126)
    assert np.all(np.abs(f64(s8) - s_ref) <= s_ref * (2 * chain(cols) + 2.0 ** -22))
    err = np.abs(f64(q8) * f64(s8)[:, None] - y_ref)
    assert np.all(err <= s_ref[:, None] * 0.5 * (1 + 2.0 ** -10) + np.abs(y_ref) * 8 * chain(cols))
    assert np.abs(f64(q8)).max() == 127

    # nothing but the codes and scales asked for: the same
    qa, sa = torch.empty_like(q8), torch.empty_like(s8)
    hip.moe_rmsnorm_int8(x, g, qa, sa, 1e-5, residual=r)
    assert torch.equal(qa, q8) and torch.equal(sa, s8)
    qa, sa = torch.empty_like(q), torch.empty_like(s)
    hip.moe_rmsnorm_fp8(x, g, qa, sa, 1e-5, residual=r)
    assert torch.equal(qa.view(I8), q.view(I8)) and torch.equal(sa, s)


def test_quantised_norm_is_the_quantiser_of_the_norm(hip):
    """Powers of two as weights and a row of power-of-two mean square: y is exact in BF16, so the
    fused codes are those of the separate quantisers."""
    rng = np.random.default_rng(5)
    x = rng.choice([-1.0, 1.0], (6, 512))  # mean square 1
    g = 2.0 ** rng.integers(-3, 4, 512)
    xd, gd = (bf16_dev(wl._to_bf16_bits(v.astype(np.float32))) for v in (x, g))
    y = torch.empty_like(xd)
    hip.moe_rmsnorm_bf16(xd, gd, y, 0.0)
    assert np.array_equal(f64(y), x * g)
    q, qr = (torch.empty((6, 512), dtype=I8, device="cuda") for _ in range(2))
    s, sr = (torch.empty(6, device="cuda") for _ in range(2))
    hip.moe_rmsnorm_int8(xd, gd, q, s, 0.0)
    hip.moe_quant_int8(y, qr, sr)
    assert torch.equal(q, qr) and torch.equal(s, sr)
    f, fr = (torch.empty((6, 512), dtype=F8, device="cuda") for _ in range(2))
    s, sr = (torch.empty((6, 4), device="cuda") for _ in range(2))
    hip.moe_rmsnorm_fp8(xd, gd, f, s, 0.0)
    hip.moe_quant_fp8(y, fr, sr)
    assert torch.equal(f.view(I8), fr.view(I8)) and torch.equal(s, sr)


@pytest.mark.parametrize("place", ["h=x", "h=residual", "y=x", "strided"])
@pytest.mark.parametrize("cols", [1024, 40000])
def test_outputs_in_place_and_strided(hip, place, cols):
    xb, rb, gb = _inputs(4, cols, cols)
    h_ref, _ = ffn.rmsnorm(_values(xb), _values(gb), 1e-5, _values(rb))
    g = bf16_dev(gb)

    def wide(bits=None):
        t = torch.full((4, cols + 24), -7.0, dtype=BF16, device="cuda")
        if bits is not None:
            t[:, :cols] = bf16_dev(bits)
        return t

    bufs = {n: wide(b) for n, b in (("x", xb), ("r", rb), ("h", None), ("y", None))}
    if place != "strided":
        bufs = {n: t[:, :cols].contiguous() for n, t in bufs.items()}
    x, r, h, y = (bufs[n][:, :cols] for n in "xrhy")
    if place == "h=x":
        h = x
    if place == "h=residual":
        h = r
    want = torch.empty((4, cols), dtype=BF16, device="cuda")
    hip.moe_rmsnorm_bf16(bf16_dev(xb), g, want, 1e-5, residual=bf16_dev(rb))
    if place == "y=x":
        y = x
    q, s = torch.empty((4, cols + 8), dtype=I8, device="cuda").fill_(3), torch.empty(4, device="cuda")
    hip.moe_rmsnorm_int8(x, g, q[:, :cols], s, 1e-5, residual=r, h=h, y=y)
    assert np.array_equal(f64(h), h_ref)
    assert torch.equal(y, want)
    assert bool((q[:, cols:] == 3).all())
    if place == "strided":
        for t in bufs.values():
            assert bool((t[:, cols:] == -7.0).all())


@pytest.mark.parametrize("scale", [1e-18, 1.0, 1e15])
def test_extreme_magnitudes(hip, scale):
    xb, _, gb = _inputs(3, 512, 9, scale)
    _, y_ref = ffn.rmsnorm(_values(xb), _values(gb), 0.0)
    y = torch.empty((3, 512), dtype=BF16, device="cuda")
    hip.moe_rmsnorm_bf16(bf16_dev(xb), bf16_dev(gb), y, 0.0)
    _check_y(f64(y), y_ref, 512)


def test_rows_that_are_not_finite_and_rows_of_zeros(hip):
    x = torch.randn(4, 256, device="cuda").to(BF16)
    x[1, 17], x[2, 3], x[3] = float("nan"), float("inf"), 0.0
    g = torch.ones(256, dtype=BF16, device="cuda")
    y, q, s = torch.empty_like(x), torch.empty((4, 256), dtype=I8, device="cuda"), torch.empty(
        4, device="cuda")
    hip.moe_rmsnorm_int8(x, g, q, s, 1e-6, y=y)
    assert bool(torch.isfinite(s[[0, 3]]).all()) and not bool(torch.isfinite(s[[1, 2]]).any())
    assert not bool(q[1:].any()) and bool(q[0].any())
    assert bool(y[1].isnan().all()) and bool(y[2, 3].isnan()) and not bool(y[3].any())
    f, fs = torch.empty((4, 256), dtype=F8, device="cuda"), torch.empty((4, 2), device="cuda")
    hip.moe_rmsnorm_fp8(x, g, f, fs, 1e-6)
    assert bool(f[1].float().isnan().all()) and not bool(f[3].float().any())
    assert bool(torch.isfinite(f[0].float()).all())
    hip.moe_quant_int8(x, q, s)
    assert bool(s[1].isnan()) and bool(s[2].isinf()) and not bool(q[1:].any())
    assert s[3].item() == 2.0 ** -126


@pytest.mark.parametrize("rows,cols", SIZES)
def test_quant_int8_bit_exact(hip, rows, cols):
    xb, _, _ = _inputs(rows, cols, rows + 7 * cols)
    x = _values(xb) * (2.0 ** np.random.default_rng(rows).integers(-130, 90, (rows, 1)))
    xb = wl._to_bf16_bits(x.astype(np.float32))
    q_ref, s_ref = ffn.quantise_int8(_values(xb))
    q, s = torch.empty((rows, cols), dtype=I8, device="cuda"), torch.empty(rows, device="cuda")
    hip.moe_quant_int8(bf16_dev(xb), q, s)
    assert np.array_equal(s.cpu().numpy(), s_ref)
    assert np.array_equal(q.cpu().numpy(), q_ref)


def test_no_rows_and_no_columns(hip):
    for rows, cols in ((0, 64), (3, 0)):
        x = torch.empty((rows, cols), dtype=BF16, device="cuda")
        g = torch.empty(cols, dtype=BF16, device="cuda")
        q, s = torch.empty((rows, cols), dtype=I8, device="cuda"), torch.empty(rows, device="cuda")
        hip.moe_rmsnorm_bf16(x, g, torch.empty_like(x))
        hip.moe_rmsnorm_int8(x, g, q, s)
        hip.moe_quant_int8(x, q, s)
    torch.cuda.synchronize()


def test_on_another_stream_and_replayed(hip):
    xb, rb, gb = _inputs(9, 640, 1)
    x, r, g = bf16_dev(xb), bf16_dev(rb), bf16_dev(gb)
    q, s, h = torch.empty((9, 640), dtype=F8, device="cuda"), torch.empty((9, 5), device="cuda"), \
        torch.empty_like(x)
    qe, se, he = torch.empty_like(q), torch.empty_like(s), torch.empty_like(h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hip.moe_rmsnorm_fp8(x, g, q, s, residual=r, h=h, stream=side)
    side.synchronize()
    hip.moe_rmsnorm_fp8(x, g, qe, se, residual=r, h=he)
    assert torch.equal(q.view(I8), qe.view(I8)) and torch.equal(s, se) and torch.equal(h, he)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hip.moe_rmsnorm_fp8(x, g, q, s, residual=r, h=h)
    for i in range(3):
        x.copy_(torch.randn(9, 640, device="cuda").to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        hip.moe_rmsnorm_fp8(x, g, qe, se, residual=r, h=he)
        torch.cuda.synchronize()
        assert torch.equal(q.view(I8), qe.view(I8)) and torch.equal(s, se) and torch.equal(h, he)

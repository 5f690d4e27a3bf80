"""The FP8 operators (moe_quant_fp8, moe_dense_gemm_fp8, moe_dense_gate_up_swiglu_fp8,
moe_w8a8_grouped_gemm, moe_w8a8_grouped_gemm_swiglu) and moe_layer_fp8 against the FP64 oracle.

Tolerances, from the arithmetic:
- Quantisation of BF16 rows, and products whose sums are exact in every order (small integer
  codes, power-of-two scales): equal bits.
- A BF16 output: half a step, 2^-8 of the value, plus the error of the FP32 sum. The FP8
  matrix cores cut each product of a group of 8 neighbouring k below 2^-13 of the group's
  largest product (7 such products a group), and every FP32 addition rounds by at most 2^-24
  of a partial sum, which the sum of magnitudes bounds.
- The SwiGLU form sums in FP32 without that cut. Its scale is off by the relative error of the
  largest value; a code by half an E4M3 step (2^-4 of the value, or half of 2^-9 scales where
  the code is subnormal) plus the value's own error.
"""

import numpy as np
import pytest
import torch

from oracle import codecs, fp8, moe

pytestmark = pytest.mark.gpu

POISON8, POISON16 = 0x55, 0x7FB1


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.view(dtype)


def _f8(codes):
    return _dev(codes, torch.float8_e4m3fn)


def _host8(t):
    return t.view(torch.uint8).cpu().numpy()


def _bf16_f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _out16(rows, cols, pad_r=2, pad_c=16):
    buf = torch.full((rows + pad_r, cols + pad_c), POISON16, dtype=torch.int16, device="cuda")
    return buf, buf.view(torch.bfloat16)[:rows, :cols]


def _out8(rows, cols, pad_r=2, pad_c=16):
    buf = torch.full((rows + pad_r, cols + pad_c), POISON8, dtype=torch.uint8, device="cuda")
    return buf, buf.view(torch.float8_e4m3fn)[:rows, :cols]


def _outs(rows, cols):
    buf = torch.full((rows + 2, fp8.blocks(cols) + 3), -7.0, device="cuda")
    return buf, buf[:rows, :fp8.blocks(cols)]


def _rest_is(buf, poison, rows, cols, written=None):
    """Everything outside [rows, cols] (and outside the ``written`` rows) keeps the poison."""
    h = buf.cpu().numpy()
    mask = np.ones(h.shape, bool)
    mask[:rows, :cols] = False
    if written is not None:
        mask[:rows][~written] = True
    return bool(np.all(h[mask] == poison))


# --------------------------------------------------------------------------- quantisation

def _bf16(values):
    return torch.from_numpy(np.asarray(values, np.float32)).to(torch.bfloat16)


def _check_quant(hip, x_bf16, pad=0):
    rows, cols = x_bf16.shape
    src = torch.full((rows, cols + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    src[:, :cols] = x_bf16.cuda()
    qb, q = _out8(rows, cols)
    sb, s = _outs(rows, cols)
    hip.moe_quant_fp8(src[:, :cols], q, s)
    want_v, want_s = fp8.quantise_rows(x_bf16.float().numpy())
    got_s = s.cpu().numpy()
    assert np.array_equal(got_s, want_s, equal_nan=True)
    got_v = codecs.e4m3fn_decode(_host8(q))
    assert np.array_equal(got_v, want_v, equal_nan=True)
    assert np.array_equal(np.signbit(got_v)[got_v == 0], np.signbit(want_v)[want_v == 0])
    assert _rest_is(qb, POISON8, rows, cols) and _rest_is(sb, -7.0, rows, fp8.blocks(cols))


@pytest.mark.parametrize("rows,cols,pad", [
    (1, 16, 0), (1, 6144, 0), (3, 272, 8), (8, 6144, 0), (17, 128, 16), (64, 112, 0),
    (257, 1008, 24), (1000, 2048, 0), (4096, 144, 0)])
def test_quant_bits(hip, rows, cols, pad):
    rng = np.random.default_rng(rows + cols)
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    _check_quant(hip, _bf16(v), pad)


def test_quant_every_mantissa_pair(hip):
    """Every BF16 mantissa over every mantissa of the group's maximum, in the binades whose
    codes are normal and subnormal: the quotient's rounding, ties among it."""
    mant = 1.0 + np.arange(128) / 128
    shifts = 2.0 ** -np.arange(1, 20, dtype=np.float64)
    v = np.concatenate([np.tile(mant * s, (128, 1)) for s in shifts], axis=1)  # [128, 19 * 128]
    v[:, ::128] = mant[:, None]  # the maximum of each group
    for e in (-130, -120, -100, 0, 100, 126):  # subnormal BF16 values among the lowest
        _check_quant(hip, _bf16(v * 2.0 ** e))
    _check_quant(hip, _bf16(-v))


def test_quant_special_values(hip):
    v = np.random.default_rng(8).standard_normal((12, 400)).astype(np.float32)
    v[0] = 0.0
    v[1, 5] = np.nan
    v[2, 7], v[2, 390] = np.inf, -np.inf
    v[3] = -0.0
    v[4] = 3.3895314e38
    v[5] = 9.2e-41  # the smallest BF16 subnormal
    v[6, :128] = 0.0
    v[7, 399] = np.nan
    v[8] = 2.0 ** -118
    _check_quant(hip, _bf16(v))


def test_quant_empty(hip):
    q = torch.empty((0, 128), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((0, 1), device="cuda")
    hip.moe_quant_fp8(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), q, s)


# ------------------------------------------------------------------------------ operands

def _int_operand(rng, rows, k, block_rows):
    """Codes of {-2, .., 2} and power-of-two scales: every FP32 sum of products is exact."""
    vals = rng.integers(-2, 3, (rows, k)).astype(np.float64)
    n_s = fp8.blocks(rows) if block_rows else rows
    scale = np.exp2(rng.integers(-1, 2, (n_s, fp8.blocks(k)))).astype(np.float32)
    return fp8.e4m3_codes(vals), scale


def _normal_operand(rng, rows, k, block_rows):
    v = rng.standard_normal((rows, k)).astype(np.float32)
    q, s = fp8.quantise_rows(v)
    if block_rows:
        s = (rng.uniform(0.5, 2, (fp8.blocks(rows), fp8.blocks(k))) / 448 / np.sqrt(k)).astype(
            np.float32)
    return fp8.e4m3_codes(q), s


def _sum_bound(a, sa, w, sw, fp8_cores):
    """Bound on |FP32 sum - exact| per output (see the module's docstring)."""
    k = a.shape[1]
    x, y = np.abs(fp8.rows_f64(a, sa)), np.abs(fp8.weight(w, sw))
    total = x @ y.T
    bound = (k + fp8.blocks(k) * 4) * 2.0 ** -24 * total
    if fp8_cores:
        # 7 cuts below 2^-13 of a group's largest product; that is at most the product of the
        # two operands' largest magnitudes in the group
        gx = np.max(x.reshape(len(x), -1, 8), axis=2)
        gy = np.max(y.reshape(len(y), -1, 8), axis=2)
        bound += 7 * 2.0 ** -13 * (gx @ gy.T)
    return bound


def _assert_bf16(got, ref, bound):
    err = np.abs(got - ref)
    lim = 2.0 ** -8 * (np.abs(ref) + bound) + bound + 2.0 ** -134
    assert np.all(np.isfinite(got))
    assert np.all(err <= lim), float(np.max(err / lim))


def _assert_quantised(codes, scale, ref, rel):
    """codes * scale against FP64 values ``ref`` whose FP32 form is off by at most ``rel`` of
    the group's largest magnitude."""
    cols = ref.shape[1]
    amax = np.stack([np.max(np.abs(ref[:, b * 128:(b + 1) * 128]), axis=1)
                     for b in range(fp8.blocks(cols))], axis=1)
    s_ref = np.maximum(amax / 448, 2.0 ** -126)
    rel_s = rel + 2.0 ** -22
    assert np.all(np.abs(scale - s_ref) <= rel_s * s_ref), float(np.max(np.abs(scale / s_ref - 1)))
    back = codecs.e4m3fn_decode(codes) * fp8.expand(scale.astype(np.float64), cols)
    full = fp8.expand(s_ref, cols)
    lim = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * full) * (1 + 2 * rel_s) + \
        448 * full * rel_s
    err = np.abs(back - ref)
    assert np.all(err <= lim), float(np.max(err / lim))


# --------------------------------------------------------------------------------- dense

# Each list reaches every tile the launcher picks among (the larger ones take thousands of rows).
DENSE = [(1, 16, 16), (1, 6144, 2048), (2, 272, 6144), (5, 48, 144), (8, 2048, 656), (12, 128, 128),
         (13, 144, 512), (17, 272, 656), (33, 1360, 1040), (40, 128, 2048), (41, 384, 272),
         (70, 400, 1040), (129, 272, 256), (256, 1024, 528), (300, 2064, 400), (515, 256, 6144),
         (1030, 1040, 144), (2100, 4112, 272), (3300, 1296, 400), (4700, 144, 400),
         (1500, 2064, 784)]


@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense_exact_sums(hip, m, n, k):
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    a, sa = _int_operand(rng, m, k, False)
    w, sw = _int_operand(rng, n, k, True)
    buf, c = _out16(m, n)
    hip.moe_dense_gemm_fp8(_f8(a), _dev(sa), _f8(w), _dev(sw), c)
    assert np.array_equal(_bf16_f64(c), codecs.round_bf16(fp8.product(a, sa, w, sw)))
    assert _rest_is(buf, POISON16, m, n)


@pytest.mark.parametrize("m,n,k", [(1, 512, 2048), (9, 272, 656), (37, 400, 1040),
                                   (300, 528, 2048), (600, 1024, 6144), (3300, 1296, 400)])
def test_dense_normal_operands(hip, m, n, k):
    rng = np.random.default_rng(m + n + k)
    a, sa = _normal_operand(rng, m, k, False)
    w, sw = _normal_operand(rng, n, k, True)
    _, c = _out16(m, n)
    ad, sad, wd, swd = _f8(a), _dev(sa), _f8(w), _dev(sw)
    hip.moe_dense_gemm_fp8(ad, sad, wd, swd, c)
    got = _bf16_f64(c)
    _assert_bf16(got, fp8.product(a, sa, w, sw), _sum_bound(a, sa, w, sw, True))
    again = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    hip.moe_dense_gemm_fp8(ad, sad, wd, swd, again)
    assert torch.equal(again, c)


def test_dense_strided_operands(hip):
    """Row strides above k on every operand; what lies between the rows is NaN."""
    rng = np.random.default_rng(9)
    m, n, k = 45, 160, 400
    a, sa = _int_operand(rng, m, k, False)
    w, sw = _int_operand(rng, n, k, True)
    pad_a, pad_w = np.full((m, k + 32), 0x7F, np.uint8), np.full((n, k + 16), 0x7F, np.uint8)
    pad_a[:, :k], pad_w[:, :k] = a, w
    pad_s = np.full((m, fp8.blocks(k) + 5), np.nan, np.float32)
    pad_s[:, :fp8.blocks(k)] = sa
    _, c = _out16(m, n)
    hip.moe_dense_gemm_fp8(_f8(pad_a)[:, :k], _dev(pad_s)[:, :fp8.blocks(k)],
                           _f8(pad_w)[:, :k], _dev(sw), c)
    assert np.array_equal(_bf16_f64(c), codecs.round_bf16(fp8.product(a, sa, w, sw)))


def test_offsets_past_32_bits(hip):
    """Operands and outputs over 4 GiB: 16 rows again and again must give the same 16 outputs."""
    rng = np.random.default_rng(40)
    times, n, k = 40000, 144, 6912
    m = 16 * times
    a, sa = _int_operand(rng, 16, k, False)
    w, sw = _int_operand(rng, n, k, True)
    want = torch.from_numpy(codecs.round_bf16(fp8.product(a, sa, w, sw))).cuda().to(torch.bfloat16)
    big_a = _dev(a).repeat(times, 1).view(torch.float8_e4m3fn)
    big_sa = _dev(sa).repeat(times, 1)
    assert big_a.numel() > 2 ** 32
    buf = torch.zeros(m, 4096, dtype=torch.bfloat16, device="cuda")
    c = buf[:, 3584:3584 + n]
    assert c.stride(0) * m * 2 > 2 ** 32
    hip.moe_dense_gemm_fp8(big_a, big_sa, _f8(w), _dev(sw), c)
    assert torch.equal(c.view(times, 16, n), want.expand(times, 16, n))
    buf.zero_()
    table = _table(hip, [(w, sw), None, (w, sw)], n, k)
    off = torch.tensor([0, m // 2, m // 2 + 16, m], dtype=torch.int32, device="cuda")
    hip.moe_w8a8_grouped_gemm(big_a, big_sa, table, off, c)
    got = c.view(times, 16, n)
    assert torch.equal(got[:times // 2], want.expand(times // 2, 16, n))
    assert not bool(got[times // 2].any())
    assert torch.equal(got[times // 2 + 1:], want.expand(times // 2 - 1, 16, n))
    del buf, c, got, big_sa
    act = big_a.view(torch.uint8)  # quantised into
    x = torch.randn(16, k, device="cuda").to(torch.bfloat16)
    xs = x.repeat(times, 1)
    scale = torch.empty(m, fp8.blocks(k), device="cuda")
    hip.moe_quant_fp8(xs, act, scale)
    q1 = torch.empty(16, k, dtype=torch.uint8, device="cuda")
    s1 = torch.empty(16, fp8.blocks(k), device="cuda")
    hip.moe_quant_fp8(x, q1, s1)
    assert torch.equal(act.view(times, 16, k), q1.expand(times, 16, k))
    assert torch.equal(scale.view(times, 16, -1), s1.expand(times, 16, s1.shape[1]))


def test_dense_nan_and_infinity_stay_in_their_row(hip):
    rng = np.random.default_rng(10)
    m, n, k = 40, 144, 400
    a, sa = _int_operand(rng, m, k, False)
    w, sw = _int_operand(rng, n, k, True)
    clean = codecs.round_bf16(fp8.product(a, sa, w, sw))
    a[3, 399] = 0x7F
    sa[17, 1] = np.inf
    sa[39, 0] = np.nan
    _, c = _out16(m, n)
    hip.moe_dense_gemm_fp8(_f8(a), _dev(sa), _f8(w), _dev(sw), c)
    got = _bf16_f64(c)
    rest = [r for r in range(m) if r not in (3, 17, 39)]
    assert np.array_equal(got[rest], clean[rest])
    assert np.all(np.isnan(got[3])) and np.all(np.isnan(got[39]))
    assert not np.any(np.isfinite(got[17]))


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 2048, 6144), (7, 144, 272), (12, 256, 512),
                                   (30, 400, 1040), (64, 128, 656), (77, 1360, 1040),
                                   (130, 272, 2048), (300, 528, 400), (2900, 272, 400),
                                   (4300, 400, 272), (3100, 1296, 400)])
def test_dense_swiglu(hip, m, n, k):
    rng = np.random.default_rng(2 * m + n + k)
    a, sa = _normal_operand(rng, m, k, False)
    gate, up = (_normal_operand(rng, n, k, True) for _ in range(2))
    # gate and up of the order of the limit, so that some are clamped
    gate, up = (gate[0], gate[1] * 448 * 4), (up[0], up[1] * 448 * 4)
    qb, q = _out8(m, n)
    sb, s = _outs(m, n)
    limit = 7.0
    args = (_f8(a), _dev(sa), _f8(gate[0]), _dev(gate[1]), _f8(up[0]), _dev(up[1]))
    hip.moe_dense_gate_up_swiglu_fp8(*args, q, s, limit)
    ref = fp8.swiglu_product(a, sa, gate, up, limit)
    _assert_quantised(_host8(q), s.cpu().numpy(), ref, _swiglu_rel(a, sa, gate, up, ref, limit))
    assert _rest_is(qb, POISON8, m, n) and _rest_is(sb, -7.0, m, fp8.blocks(n))
    q2, s2 = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(s)
    hip.moe_dense_gate_up_swiglu_fp8(*args, q2, s2, limit)
    assert np.array_equal(_host8(q2), _host8(q)) and torch.equal(s2, s)


@pytest.mark.parametrize("m,n,k", [(1, 2048, 6144), (8, 272, 2048), (40, 144, 2064),
                                   (200, 400, 2064)])
def test_dense_swiglu_split_over_k(hip, m, n, k):
    """Sizes that split K: through a workspace of the caller's, through the call's own (same
    bits), nothing written past it, and a workspace that is too small is refused."""
    need = hip.moe_fp8_swiglu_workspace_bytes(m, 0, n, k)
    assert need > 0 and need % (m * n * 8) == 0
    rng = np.random.default_rng(m + n)
    a, sa = _normal_operand(rng, m, k, False)
    gate, up = (_normal_operand(rng, n, k, True) for _ in range(2))
    gate, up = (gate[0], gate[1] * 448 * 4), (up[0], up[1] * 448 * 4)
    args = (_f8(a), _dev(sa), _f8(gate[0]), _dev(gate[1]), _f8(up[0]), _dev(up[1]))
    qb, q = _out8(m, n)
    sb, s = _outs(m, n)
    buf = torch.full((need + 512,), 0x6B, dtype=torch.uint8, device="cuda")
    hip.moe_dense_gate_up_swiglu_fp8(*args, q, s, 7.0, workspace=buf[:need])
    ref = fp8.swiglu_product(a, sa, gate, up, 7.0)
    _assert_quantised(_host8(q), s.cpu().numpy(), ref, _swiglu_rel(a, sa, gate, up, ref, 7.0))
    assert bool(torch.all(buf[need:] == 0x6B))
    assert _rest_is(qb, POISON8, m, n) and _rest_is(sb, -7.0, m, fp8.blocks(n))
    q2, s2 = torch.empty((m, n), dtype=q.dtype, device="cuda"), torch.empty_like(s)
    hip.moe_dense_gate_up_swiglu_fp8(*args, q2, s2, 7.0)
    assert np.array_equal(_host8(q2), _host8(q)) and torch.equal(s2, s)
    q2.view(torch.uint8).fill_(POISON8)
    with pytest.raises(hip.MoeError) as err:
        hip.moe_dense_gate_up_swiglu_fp8(*args, q2, s2, 7.0, workspace=buf[:need - 16])
    assert err.value.status == 2
    torch.cuda.synchronize()
    assert bool(torch.all(q2.view(torch.uint8) == POISON8))


def test_dense_swiglu_split_on_another_stream(hip):
    """The call's own workspace belongs to the given stream: two chains on two streams."""
    rng = np.random.default_rng(31)
    m, n, k = 16, 512, 2048
    assert hip.moe_fp8_swiglu_workspace_bytes(m, 0, n, k) > 0
    jobs = []
    for _ in range(2):
        a, sa = _normal_operand(rng, m, k, False)
        g, u = (_normal_operand(rng, n, k, True) for _ in range(2))
        args = (_f8(a), _dev(sa), _f8(g[0]), _dev(g[1]), _f8(u[0]), _dev(u[1]))
        outs = [(torch.empty((m, n), dtype=torch.float8_e4m3fn, device="cuda"),
                 torch.empty((m, fp8.blocks(n)), device="cuda")) for _ in range(2)]
        hip.moe_dense_gate_up_swiglu_fp8(*args, *outs[0], 7.0)
        jobs.append((args, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for args, outs, st in jobs:
            hip.moe_dense_gate_up_swiglu_fp8(*args, *outs[1], 7.0, stream=st)
    torch.cuda.synchronize()
    for _, outs, _ in jobs:
        assert np.array_equal(_host8(outs[0][0]), _host8(outs[1][0]))
        assert torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("k", [16, 2064])
def test_dense_swiglu_far_negative_gates(hip, k):
    """silu down to where e^g leaves the FP32 numbers, lifted by large up values. The gates are
    exact. e^-|g| is off by |g| times the rounding of the exponent (2^-24, its 64 added 2^-24,
    the constant 2^-26), by an ulp of the exponential and half a subnormal step; the
    reciprocal by an ulp, the sum, three products and the scale's division by 2^-24 each."""
    gates = np.array([1, 20, 60, 80, 86.5, 87.25, 88, 90, 95, 100, 103, 104, 120, 1000], np.float32)
    m, n = len(gates), 144
    a = np.zeros((m, k), np.uint8)
    a[:, 0] = 0x38  # 1.0
    sa = np.ones((m, fp8.blocks(k)), np.float32)
    sa[:, 0] = gates
    gate, up = np.zeros((n, k), np.uint8), np.zeros((n, k), np.uint8)
    gate[:, 0], up[:, 0] = 0xB8, 0x38
    one = np.ones((fp8.blocks(n), fp8.blocks(k)), np.float32)
    q = torch.empty((m, n), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((m, fp8.blocks(n)), device="cuda")
    hip.moe_dense_gate_up_swiglu_fp8(_f8(a), _dev(sa), _f8(gate), _dev(one), _f8(up),
                                     _dev(one * np.float32(2.0 ** 100)), q, s, 3e38)
    g = gates.astype(np.float64)
    u = g * 2.0 ** 100
    v = g * np.exp(-g) / (1 + np.exp(-g)) * u
    bound = v * (2.25 * g + 10) * 2.0 ** -24 + (g + 1) * 2.0 ** -150 * u
    got = s.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - (v / 448)[:, None]) <= (bound / 448 + 2.0 ** -126)[:, None])
    codes = _host8(q)
    assert np.all(codes[g <= 100] == 0xFE)  # -448, the group's largest
    assert np.all(codes[g >= 110] & 0x7F == 0)


def _swiglu_rel(a, sa, gate, up, ref, limit):
    """The largest error of v = silu(G) U in FP32, relative to its group's largest |v|: the
    sums' errors times the partial derivatives (|silu'| <= 1.1, |U| <= limit, |silu(G)| <=
    limit) plus 2^-20 of v for the exponential and the arithmetic."""
    err = 1.1 * limit * _sum_bound(a, sa, *gate, False) + limit * _sum_bound(a, sa, *up, False)
    cols = ref.shape[1]
    worst = 0.0
    for b in range(fp8.blocks(cols)):
        c = slice(b * 128, min((b + 1) * 128, cols))
        amax = np.max(np.abs(ref[:, c]), axis=1, keepdims=True)
        worst = max(worst, float(np.max(err[:, c] / np.maximum(amax, 1e-30))))
    return worst + 2.0 ** -20


# ------------------------------------------------------------------------------- grouped

def _table(hip, experts, n, k, gate_up=False):
    return hip.Fp8ExpertTable([None if e is None else _f8(e[0]) for e in experts],
                              [None if e is None else _dev(e[1]) for e in experts], n, k,
                              gate_up=gate_up, device="cuda:0")


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _counts(rng, experts, total, kind):
    if kind == "even":
        p = np.ones(experts)
    else:
        p = 1.0 / (1 + rng.permutation(experts)) ** 1.5
    c = rng.multinomial(total, p / p.sum())
    if experts > 2:  # an expert without rows, between others
        c[1] += c[experts // 2]
        c[experts // 2] = 0
    return c


GROUPED = [  # experts, rows, n, k, counts
    (1, 1, 16, 16, "even"), (4, 3, 272, 144, "even"), (9, 21, 272, 656, "skew"),
    (16, 130, 144, 512, "even"), (16, 513, 400, 272, "skew"), (64, 100, 256, 256, "skew"),
    (70, 2000, 128, 400, "skew"), (8, 700, 1040, 528, "even"), (130, 260, 160, 128, "even"),
    (3, 1500, 272, 1040, "skew"), (2048, 300, 32, 48, "even"), (5, 1100, 528, 400, "even"),
    (8, 4800, 144, 400, "skew"), (12, 3387, 1040, 400, "skew"), (12, 3600, 1040, 272, "even")]


@pytest.mark.parametrize("experts,rows,n,k,kind", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_exact_sums(hip, experts, rows, n, k, kind, gather):
    rng = np.random.default_rng(experts + rows + n + k)
    off = _offsets(_counts(rng, experts, rows, kind))
    a_rows = max(rows // 3, 1) if gather else rows
    a, sa = _int_operand(rng, a_rows, k, False)
    idx = rng.integers(0, a_rows, rows).astype(np.int32)
    if gather and rows > 10:
        idx[[0, rows // 2, rows - 1]] = [-1, a_rows, 2 ** 30]  # out of range: zeros
    weights = [None if (experts > 3 and e % 5 == 3) else _int_operand(rng, n, k, True)
               for e in range(experts)]
    buf, c = _out16(rows, n)
    hip.moe_w8a8_grouped_gemm(_f8(a), _dev(sa), _table(hip, weights, n, k), _dev(off), c,
                              a_gather=_dev(idx) if gather else None)
    got, written = _bf16_f64(c), np.zeros(rows, bool)
    for e, lo, hi in fp8.segments(off, rows):
        if weights[e] is None:
            continue
        written[lo:hi] = True
        src = fp8.gathered(a, sa, idx[lo:hi]) if gather else (a[lo:hi], sa[lo:hi])
        want = codecs.round_bf16(fp8.product(*src, *weights[e]))
        assert np.array_equal(got[lo:hi], want), f"expert {e}, rows {lo}..{hi}"
    assert _rest_is(buf, POISON16, rows, n, written)


def test_grouped_row_cut(hip):
    """max_rows below the slots: rows from it on keep their values, also inside a tile."""
    rng = np.random.default_rng(12)
    experts, rows, n, k = 6, 200, 144, 272
    off = _offsets([50, 0, 90, 20, 40, 0])
    a, sa = _int_operand(rng, rows, k, False)
    weights = [_int_operand(rng, n, k, True) for _ in range(experts)]
    table = _table(hip, weights, n, k)
    for cut in (0, 1, 49, 50, 51, 139, 145, 199):
        buf, c = _out16(rows, n)
        hip.moe_w8a8_grouped_gemm(_f8(a), _dev(sa), table, _dev(off), c, max_rows=cut)
        got = _bf16_f64(c)
        for e, lo, hi in fp8.segments(off, cut):
            want = codecs.round_bf16(fp8.product(a[lo:hi], sa[lo:hi], *weights[e]))
            assert np.array_equal(got[lo:hi], want)
        assert _rest_is(buf, POISON16, cut, n)


@pytest.mark.parametrize("off", [[0, 40, 20, 60, 60], [5, 5, -3, 70, 10], [0, 0, 0, 0, 0],
                                 [60, 30, 20, 10, 0], [-10, 20, 2000000000, 40, 60]])
def test_grouped_offsets_that_are_no_prefix_sum_stay_in_range(hip, off):
    """Such offsets miss or repeat rows; nothing outside the output's rows is written."""
    rng = np.random.default_rng(13)
    rows, n, k = 60, 144, 144
    a, sa = _int_operand(rng, rows, k, False)
    table = _table(hip, [_int_operand(rng, n, k, True) for _ in range(4)], n, k)
    buf, c = _out16(rows, n)
    hip.moe_w8a8_grouped_gemm(_f8(a), _dev(sa), table, _dev(np.array(off, np.int32)), c)
    torch.cuda.synchronize()
    assert _rest_is(buf, POISON16, rows, n)


@pytest.mark.parametrize("experts,n", [(300, 144), (2048, 16), (70, 2064)])
def test_grouped_experts_of_every_size(hip, experts, n):
    """Counts from none to several tiles in no order, some experts absent: the work goes by size."""
    rng = np.random.default_rng(experts)
    k = 144
    counts = np.where(rng.random(experts) < 0.3, 0, np.exp(rng.uniform(0, 4.5, experts)))
    counts = counts.astype(np.int64)
    counts[experts // 3] = 700
    off = _offsets(counts)
    rows = int(off[-1])
    a, sa = _int_operand(rng, rows, k, False)
    pool = [_int_operand(rng, n, k, True) for _ in range(7)]
    weights = [None if e % 11 == 5 else pool[e % 7] for e in range(experts)]
    buf, c = _out16(rows, n)
    hip.moe_w8a8_grouped_gemm(_f8(a), _dev(sa), _table(hip, weights, n, k), _dev(off), c)
    got, written = _bf16_f64(c), np.zeros(rows, bool)
    for e, lo, hi in fp8.segments(off, rows):
        if weights[e] is not None:
            written[lo:hi] = True
            want = codecs.round_bf16(fp8.product(a[lo:hi], sa[lo:hi], *weights[e]))
            assert np.array_equal(got[lo:hi], want), e
    assert _rest_is(buf, POISON16, rows, n, written)


GROUPED_SWIGLU = [  # experts, tokens, top_k, mi, k, counts
    (1, 1, 1, 16, 16, "even"), (8, 3, 2, 128, 272, "even"), (9, 33, 3, 272, 656, "skew"),
    (16, 65, 4, 144, 512, "even"), (16, 300, 4, 400, 272, "skew"), (64, 20, 8, 256, 256, "skew"),
    (4, 500, 2, 272, 1040, "skew"), (6, 400, 3, 160, 400, "even"), (40, 900, 2, 144, 272, "skew"),
    (20, 1902, 2, 144, 400, "skew"), (20, 1630, 3, 400, 400, "skew"), (17, 2400, 1, 784, 400, "even"),
    (5, 120, 2, 4112, 144, "skew"), (70, 4500, 2, 272, 272, "even")]


@pytest.mark.parametrize("experts,tokens,top_k,mi,k,kind", GROUPED_SWIGLU)
def test_grouped_swiglu(hip, experts, tokens, top_k, mi, k, kind):
    rng = np.random.default_rng(experts + tokens + mi + k)
    rows = tokens * top_k
    off = _offsets(_counts(rng, experts, rows, kind))
    a, sa = _normal_operand(rng, tokens, k, False)
    idx = rng.integers(0, tokens, rows).astype(np.int32)
    if rows > 10:
        idx[rows // 2] = tokens  # zeros: codes 0, the smallest scale

    def fused():
        g, u = (_normal_operand(rng, mi, k, True) for _ in range(2))
        return np.concatenate([g[0], u[0]]), np.concatenate([g[1], u[1]]) * np.float32(448 * 4)

    weights = [None if (experts > 3 and e % 5 == 3) else fused() for e in range(experts)]
    qb, q = _out8(rows, mi)
    sb, s = _outs(rows, mi)
    limit = 7.0
    hip.moe_w8a8_grouped_gemm_swiglu(_f8(a), _dev(sa), _table(hip, weights, 2 * mi, k, True),
                                     _dev(off), q, s, limit, a_gather=_dev(idx))
    codes, scale, written = _host8(q), s.cpu().numpy(), np.zeros(rows, bool)
    for e, lo, hi in fp8.segments(off, rows):
        if weights[e] is None:
            continue
        written[lo:hi] = True
        src = fp8.gathered(a, sa, idx[lo:hi])
        gate, up = fp8.split_gate_up(*weights[e])
        ref = fp8.swiglu_product(*src, gate, up, limit)
        live = np.any(ref != 0, axis=1)
        assert np.all(codes[lo:hi][~live] & 0x7F == 0)
        assert np.all(scale[lo:hi][~live] == np.float32(2.0 ** -126))
        if live.any():
            src = (src[0][live], src[1][live])
            _assert_quantised(codes[lo:hi][live], scale[lo:hi][live], ref[live],
                              _swiglu_rel(*src, gate, up, ref[live], limit))
    assert _rest_is(qb, POISON8, rows, mi, written)
    assert _rest_is(sb, -7.0, rows, fp8.blocks(mi), written)


@pytest.mark.parametrize("k", [16, 112, 128, 240])
def test_few_k_on_large_tiles(hip, k):
    """Fewer steps than the large tiles have stages: one block of k, one that is partial, two."""
    test_dense_exact_sums(hip, 4200, 2064, k)
    test_dense_swiglu(hip, 4300, 400, k)
    test_grouped_exact_sums(hip, 6, 3000, 2064, k, "skew", True)
    test_grouped_swiglu(hip, 70, 4500, 2, 272, k, "even")


def test_grouped_swiglu_split_leaves_uncovered_rows(hip):
    """The split form's second launch writes the rows of present experts only."""
    rng = np.random.default_rng(33)
    experts, rows, mi, k = 6, 24, 144, 2064
    off = _offsets([5, 0, 4, 6, 2, 3])  # rows 20.. belong to nobody
    assert hip.moe_fp8_swiglu_workspace_bytes(rows, experts, mi, k) > 0
    a, sa = _normal_operand(rng, rows, k, False)
    weights = []
    for e in range(experts):
        g, u = (_normal_operand(rng, mi, k, True) for _ in range(2))
        weights.append(None if e in (2, 5) else (np.concatenate([g[0], u[0]]),
                                                 np.concatenate([g[1], u[1]]) * np.float32(448)))
    qb, q = _out8(rows, mi)
    sb, s = _outs(rows, mi)
    hip.moe_w8a8_grouped_gemm_swiglu(_f8(a), _dev(sa), _table(hip, weights, 2 * mi, k, True),
                                     _dev(off), q, s, 7.0)
    written = np.zeros(rows, bool)
    for e, lo, hi in fp8.segments(off, rows):
        if weights[e] is None:
            continue
        written[lo:hi] = True
        gate, up = fp8.split_gate_up(*weights[e])
        ref = fp8.swiglu_product(a[lo:hi], sa[lo:hi], gate, up, 7.0)
        _assert_quantised(_host8(q)[lo:hi], s.cpu().numpy()[lo:hi], ref,
                          _swiglu_rel(a[lo:hi], sa[lo:hi], gate, up, ref, 7.0))
    assert _rest_is(qb, POISON8, rows, mi, written)
    assert _rest_is(sb, -7.0, rows, fp8.blocks(mi), written)


def test_swiglu_nan_and_infinity_stay_in_their_row(hip):
    rng = np.random.default_rng(14)
    m, n, k = 20, 160, 272
    a, sa = _int_operand(rng, m, k, False)
    gate, up = _int_operand(rng, n, k, True), _int_operand(rng, n, k, True)

    def call(a, sa):
        q = torch.empty((m, n), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((m, fp8.blocks(n)), device="cuda")
        hip.moe_dense_gate_up_swiglu_fp8(_f8(a), _dev(sa), _f8(gate[0]), _dev(gate[1]),
                                         _f8(up[0]), _dev(up[1]), q, s, 7.0)
        return _host8(q), s.cpu().numpy()

    q0, s0 = call(a, sa)
    a2, sa2 = a.copy(), sa.copy()
    a2[4, 100] = 0xFF
    sa2[9, 2] = np.nan
    q1, s1 = call(a2, sa2)
    rest = [r for r in range(m) if r not in (4, 9)]
    assert np.array_equal(q1[rest], q0[rest]) and np.array_equal(s1[rest], s0[rest])
    assert np.all(np.isnan(s1[[4, 9]])) and np.all(q1[[4, 9]] & 0x7F == 0x7F)


# --------------------------------------------------------------------------------- layer

def _layer(hip, seed, rows, experts, top_k, hidden, mi, absent=(), shared=False, max_rows=None):
    rng = np.random.default_rng(seed)
    gu, dn = [], []
    for e in range(experts):
        if e in absent:
            gu.append(None)
            dn.append(None)
            continue
        g, u = (_normal_operand(rng, mi, hidden, True) for _ in range(2))
        gu.append((np.concatenate([g[0], u[0]]),
                   np.concatenate([g[1], u[1]]) * np.float32(448)))
        d = _normal_operand(rng, hidden, mi, True)
        dn.append((d[0], d[1] * np.float32(448)))
    sh = None
    if shared:
        sh = [(w[0], w[1] * np.float32(448)) for w in
              (_normal_operand(rng, mi, hidden, True), _normal_operand(rng, mi, hidden, True),
               _normal_operand(rng, hidden, mi, True))]
    tables = _table(hip, gu, 2 * mi, hidden, True), _table(hip, dn, hidden, mi)
    ws = hip.Fp8Workspace(max_rows or rows, top_k, experts, hidden, mi)
    shared_hip = None
    if shared:
        flat = [t for w in sh for t in (_f8(w[0]), _dev(w[1]))]
        shared_hip = hip.SharedExpertFp8(*flat, max_rows or rows)
    return rng, gu, dn, sh, tables, ws, shared_hip


def _layer_inputs(rng, rows, experts, top_k, hidden):
    x = _bf16(rng.standard_normal((rows, hidden)))
    ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(rows)]).astype(np.int32)
    w = rng.uniform(0.1, 1, (rows, top_k)).astype(np.float32)
    return x, ids, w / w.sum(1, keepdims=True)


@pytest.mark.parametrize("rows,experts,top_k,hidden,mi,absent,shared", [
    (1, 8, 2, 256, 128, (), False), (5, 6, 3, 272, 144, (2,), False),
    (40, 16, 4, 512, 256, (0, 7), True), (200, 4, 2, 384, 400, (), True)])
def test_layer_vs_oracle(hip, rows, experts, top_k, hidden, mi, absent, shared):
    rng, gu, dn, sh, (gt, dt), ws, sh_hip = _layer(hip, rows, rows, experts, top_k, hidden, mi,
                                                   absent, shared)
    x, ids, w = _layer_inputs(rng, rows, experts, top_k, hidden)
    if rows > 4:
        ids[2, 1] = -1  # an unfilled router slot
    out = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda")
    hip.moe_layer_fp8(x.cuda(), _dev(ids), _dev(w), gt, dt, 7.0, ws, out, sh_hip)
    x32 = x.float().numpy()
    shared_ref = None
    if shared:
        v, s = fp8.quantise_rows(x32)
        act = fp8.swiglu_product(fp8.e4m3_codes(v), s, sh[0], sh[1], 7.0)
        av, as_ = fp8.quantise_rows(act.astype(np.float32))
        shared_ref = codecs.round_bf16(fp8.product(fp8.e4m3_codes(av), as_, *sh[2]))
    ref = fp8.moe_layer(x32, ids, w, gu, dn, 7.0, shared_ref)
    got = _bf16_f64(out)
    # Codes of the activation may differ by one E4M3 step (2^-3) where its FP32 value lies
    # next to a border, which for values whose error is below 2^-18 of them happens to fewer
    # than one in 2^11; a row's output then moves by at most 2^-3 of one term of a sum of mi.
    # The rest is two BF16 roundings. All of it stays below 2^-6 of the row's largest output.
    top = np.max(np.abs(ref), axis=1, keepdims=True)
    assert np.all(np.abs(got - ref) <= 2.0 ** -6 * top), float(np.max(np.abs(got - ref) / top))
    assert np.linalg.norm(got - ref) <= 2.0 ** -7 * np.linalg.norm(ref)


def test_layer_is_its_calls_in_turn(hip):
    rows, experts, top_k, hidden, mi = 70, 12, 3, 384, 272
    rng, _, _, _, (gt, dt), ws, _ = _layer(hip, 20, rows, experts, top_k, hidden, mi)
    x, ids, w = _layer_inputs(rng, rows, experts, top_k, hidden)
    x, ids, w = x.cuda(), _dev(ids), _dev(w)
    out = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda")
    hip.moe_layer_fp8(x, ids, w, gt, dt, 7.0, ws, out)
    q = torch.empty((rows, hidden), dtype=torch.float8_e4m3fn, device="cuda")
    qs = torch.empty((rows, fp8.blocks(hidden)), device="cuda")
    hip.moe_quant_fp8(x, q, qs)
    s = rows * top_k
    act = torch.empty((s, mi), dtype=torch.float8_e4m3fn, device="cuda")
    act_s = torch.empty((s, fp8.blocks(mi)), device="cuda")
    order = torch.argsort(ids.view(-1), stable=True)
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(ids.view(-1), minlength=experts).cumsum(0)
    hip.moe_w8a8_grouped_gemm_swiglu(q, qs, gt, off, act, act_s, 7.0,
                                     a_gather=(order // top_k).int())
    y = torch.empty((s, hidden), dtype=torch.bfloat16, device="cuda")
    hip.moe_w8a8_grouped_gemm(act, act_s, dt, off, y)
    perm = torch.empty(s, dtype=torch.int32, device="cuda")
    perm[order] = torch.arange(s, dtype=torch.int32, device="cuda")
    want = torch.empty_like(out)
    hip.moe_combine(y, perm, w, want)
    assert torch.equal(out, want)


def test_expert_parallel_halves_sum_to_the_whole(hip):
    """Two tables with complementary null entries: their layers' outputs add up."""
    rows, experts, top_k, hidden, mi = 24, 8, 4, 256, 128
    rng, gu, dn, _, (gt, dt), ws, _ = _layer(hip, 21, rows, experts, top_k, hidden, mi)
    x, ids, w = _layer_inputs(rng, rows, experts, top_k, hidden)
    x, ids, w = x.cuda(), _dev(ids), _dev(w)
    outs = []
    for keep in (range(experts), range(4), range(4, 8)):
        g = _table(hip, [gu[e] if e in keep else None for e in range(experts)], 2 * mi, hidden, True)
        d = _table(hip, [dn[e] if e in keep else None for e in range(experts)], hidden, mi)
        out = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda")
        hip.moe_layer_fp8(x, ids, w, g, d, 7.0, ws, out)
        outs.append(_bf16_f64(out))
    # three BF16 roundings of values no larger than the largest partial sum
    top = np.max(np.abs(np.stack(outs)))
    assert np.max(np.abs(outs[0] - outs[1] - outs[2])) <= 3 * 2.0 ** -8 * top


def test_layer_captured_and_replayed(hip):
    rows, experts, top_k, hidden, mi = 33, 10, 2, 256, 160
    rng, _, _, _, (gt, dt), ws, sh = _layer(hip, 22, rows, experts, top_k, hidden, mi, (3,), True)
    bufs = None
    inputs = [_layer_inputs(rng, rows, experts, top_k, hidden) for _ in range(4)]
    x, ids, w = inputs[0][0].cuda(), _dev(inputs[0][1]), _dev(inputs[0][2])
    out = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda")
    bufs = (x, ids, w)
    hip.moe_layer_fp8(*bufs, gt, dt, 7.0, ws, out, sh)  # every attribute set before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        hip.moe_layer_fp8(*bufs, gt, dt, 7.0, ws, out, sh)
    for xi, idi, wi in inputs[1:] + inputs[:1]:
        x.copy_(xi.cuda())
        ids.copy_(_dev(idi))
        w.copy_(_dev(wi))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = torch.empty_like(out)
        ws2 = hip.Fp8Workspace(rows, top_k, experts, hidden, mi)
        hip.moe_layer_fp8(*bufs, gt, dt, 7.0, ws2, eager, sh)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)


def test_layer_with_a_bf16_shared_term_and_without_rows(hip):
    """The shared term as a BF16 SharedExpert and as a tensor give the same bits; no rows
    enqueue nothing."""
    rows, experts, top_k, hidden, mi = 20, 6, 2, 256, 128
    rng, _, _, _, (gt, dt), ws, _ = _layer(hip, 24, rows, experts, top_k, hidden, mi)
    x, ids, w = _layer_inputs(rng, rows, experts, top_k, hidden)
    x, ids, w = x.cuda(), _dev(ids), _dev(w)
    g, u, d = (_bf16(rng.standard_normal(s) / 16).cuda() for s in ((64, hidden), (64, hidden),
                                                                   (hidden, 64)))
    sh = hip.SharedExpert(g, u, d, rows)
    outs = [torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    hip.moe_layer_fp8(x, ids, w, gt, dt, 7.0, ws, outs[0], sh)
    hip.moe_layer_fp8(x, ids, w, gt, dt, 7.0, ws, outs[1], sh(x, 7.0))
    assert torch.equal(outs[0], outs[1])
    hip.moe_layer_fp8(x[:0], ids[:0], w[:0], gt, dt, 7.0, ws, outs[1][:0])
    with pytest.raises(ValueError):
        hip.moe_layer_fp8(x, ids, w, gt, dt, 7.0, hip.Fp8Workspace(rows, 3, experts, hidden, mi),
                          outs[0])
    with pytest.raises(ValueError):
        hip.moe_layer_fp8(x, ids, w, dt, gt, 7.0, ws, outs[0])


def test_calls_run_on_the_given_stream(hip):
    """Two independent chains on two streams, each with its own buffers."""
    rng = np.random.default_rng(23)
    m, n, k = 64, 256, 512
    jobs = []
    for _ in range(2):
        a, sa = _int_operand(rng, m, k, False)
        w, sw = _int_operand(rng, n, k, True)
        jobs.append(([_f8(a), _dev(sa), _f8(w), _dev(sw)],
                     torch.zeros((m, n), dtype=torch.bfloat16, device="cuda"),
                     codecs.round_bf16(fp8.product(a, sa, w, sw)), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for args, c, _, st in jobs:
            hip.moe_dense_gemm_fp8(*args, c, stream=st)
    torch.cuda.synchronize()
    for _, c, want, _ in jobs:
        assert np.array_equal(_bf16_f64(c), want)


# ------------------------------------------------------------------------------ refusals

def test_binding_refuses(hip):
    f8 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    a, sa = torch.zeros((4, 256), **f8), torch.ones((4, 2), device="cuda")
    w, sw = torch.zeros((144, 256), **f8), torch.ones((2, 2), device="cuda")
    c = torch.zeros((4, 144), dtype=torch.bfloat16, device="cuda")
    hip.moe_dense_gemm_fp8(a, sa, w, sw, c)
    with pytest.raises(TypeError):
        hip.moe_dense_gemm_fp8(a.float(), sa, w, sw, c)
    with pytest.raises(TypeError):
        hip.moe_dense_gemm_fp8(a, sa.double(), w, sw, c)
    with pytest.raises(ValueError):
        hip.moe_dense_gemm_fp8(a, sa[:, :1], w, sw, c)
    with pytest.raises(ValueError):
        hip.moe_dense_gemm_fp8(a, sa, w, sw[:1], c)
    with pytest.raises(ValueError):
        hip.moe_dense_gemm_fp8(a, sa, w, sw, c[:, :128])
    with pytest.raises(ValueError):
        hip.moe_dense_gemm_fp8(a, sa, w[:, :128], sw, c)
    with pytest.raises(TypeError):
        hip.moe_dense_gemm_fp8(a, sa.cpu(), w, sw, c)
    with pytest.raises(hip.MoeError):  # k not a multiple of 16
        hip.moe_dense_gemm_fp8(a[:, :250], sa, w[:, :250], sw, c)
    table = hip.Fp8ExpertTable([w], [sw], 144, 256)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        hip.moe_w8a8_grouped_gemm_swiglu(a, sa, table, off, a, sa, 7.0)
    with pytest.raises(ValueError):
        hip.moe_w8a8_grouped_gemm(a, sa, table, off[:1], c)
    with pytest.raises(ValueError):
        hip.moe_w8a8_grouped_gemm(a, sa, table, off, c, max_rows=5)
    with pytest.raises(ValueError):
        hip.Fp8ExpertTable([w], [sw], 144, 256, gate_up=False, device="cpu")
    with pytest.raises(ValueError):
        hip.Fp8ExpertTable([w, None], [sw, sw], 144, 256)
    with pytest.raises(ValueError):
        hip.Fp8ExpertTable([w], [sw[:1]], 144, 256)
    q = torch.zeros((4, 144), **f8)
    with pytest.raises(ValueError):
        hip.moe_quant_fp8(c, q, torch.ones((4, 1), device="cuda"))
    with pytest.raises(ValueError):
        hip.moe_quant_fp8(c, q[:3], torch.ones((4, 2), device="cuda"))

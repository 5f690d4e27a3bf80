"""The INT8 products against the oracle. The sums are exact and the FP32 steps behind them are
defined, so the plain product is compared bit for bit. The SwiGLU form adds its exponential: off
by (|g| + 8) 2^-24 of the result at most, |g| <= 104 before the result is below 2^-120; with the
BF16 rounding 2^-8 + 2^-17 of the value."""

import numpy as np
import pytest
import torch

from gpu_util import bf16_dev, dev, f64
import workloads as wl
from oracle import codecs, ffn

pytestmark = pytest.mark.gpu
BF16, I8 = torch.bfloat16, torch.int8


def _codes(rng, rows, k, lo=-127):
    return rng.integers(lo, 128, (rows, k)).astype(np.int8)


def _scales(rng, n):
    return (rng.random(n) + 0.01).astype(np.float32) / 1000


def _wide(codes, pad=32):
    """The codes as a view of a wider device buffer."""
    t = torch.full((codes.shape[0], codes.shape[1] + pad), 99, dtype=I8, device="cuda")
    t[:, :codes.shape[1]] = dev(codes)
    return t[:, :codes.shape[1]]


# every kernel and tile: one row, the few-row kernels' edges, ragged rows and columns, one k step,
# k past a step's end, many tiles
SIZES = [(1, 16, 16), (1, 6144, 2048), (2, 48, 144), (16, 272, 1040), (17, 96, 256), (32, 160, 2064),
         (33, 48, 384), (64, 1360, 1040), (65, 144, 128), (77, 1360, 1040), (128, 256, 400),
         (256, 528, 2048), (300, 272, 720), (512, 144, 16), (513, 400, 1168), (700, 1040, 528),
         (1024, 768, 640), (1500, 2064, 272), (2049, 272, 144), (4096, 512, 256), (40, 4112, 272),
         (139, 5648, 144), (556, 6752, 144), (1121, 6768, 144), (1559, 7088, 144), (2689, 2256, 288)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_dense_bit_exact(hip, m, n, k):
    rng = np.random.default_rng(m + n + k)
    a, w, sa, sw = _codes(rng, m, k, -128), _codes(rng, n, k, -128), _scales(rng, m), _scales(rng, n)
    c = torch.full((m + 2, n + 8), 5.0, dtype=BF16, device="cuda")
    view = c[:m, :n]
    hip.moe_dense_gemm_int8(_wide(a), dev(sa), _wide(w, 16), dev(sw), view)
    assert np.array_equal(f64(view), ffn.int8_product(a, sa, w, sw))
    assert bool((c[m:] == 5.0).all()) and bool((c[:, n:] == 5.0).all())


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("limit", [7.0, 0.5])
def test_swiglu(hip, m, n, k, limit):
    rng = np.random.default_rng(m * n + k)
    a, g, u = _codes(rng, m, k), _codes(rng, n, k), _codes(rng, n, k)
    # gate and up of a few units: inside the clamp and past it
    sa, sg, su = (rng.random(s).astype(np.float32) + 0.5 for s in (m, n, n))
    sa /= np.float32(2000 * np.sqrt(k))
    act = torch.full((m + 1, n + 4), 5.0, dtype=BF16, device="cuda")
    view = act[:m, :n]
    hip.moe_dense_gate_up_swiglu_int8(_wide(a), dev(sa), _wide(g), dev(sg), _wide(u), dev(su),
                                      view, limit)
    ref = ffn.int8_swiglu(a, sa, g, sg, u, su, limit)
    assert np.all(np.abs(f64(view) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -17) + 2.0 ** -120)
    assert bool((act[m:] == 5.0).all()) and bool((act[:, n:] == 5.0).all())


def test_longest_sums(hip):
    k = hip.INT8_MAX_K
    for m in (1, 70, 600):
        a, w = np.full((m, k), -128, np.int8), np.full((16, k), -128, np.int8)
        w[3], w[5] = 127, 0
        one = np.ones(m, np.float32)
        c = torch.empty((m, 16), dtype=BF16, device="cuda")
        hip.moe_dense_gemm_int8(dev(a), dev(one), dev(w), dev(one[:1].repeat(16)), c)
        assert np.array_equal(f64(c), ffn.int8_product(a, one, w, one[:1].repeat(16)))


def test_scales_that_are_not_finite_stay_in_their_row_and_column(hip):
    rng = np.random.default_rng(0)
    for m in (5, 90, 600):
        a, w = _codes(rng, m, 256), _codes(rng, 48, 256)
        sa, sw = _scales(rng, m), _scales(rng, 48)
        sa[2], sw[7] = np.nan, np.inf
        a[2] = 0
        c = torch.empty((m, 48), dtype=BF16, device="cuda")
        hip.moe_dense_gemm_int8(dev(a), dev(sa), dev(w), dev(sw), c)
        got = f64(c)
        assert np.isnan(got[2]).all() and not np.isfinite(got[:, 7]).any()
        keep = np.ix_(np.arange(m) != 2, np.arange(48) != 7)
        assert np.array_equal(got[keep], ffn.int8_product(a, sa, w, sw)[keep])


def _expert(rng, inter, hidden):
    w = [(_codes(rng, r, k), ((rng.random(r) + 0.5) / (60 * np.sqrt(k))).astype(np.float32))
         for r, k in ((inter, hidden), (inter, hidden), (hidden, inter))]
    return w, [dev(t) for p in w for t in p]


@pytest.mark.parametrize("rows,hidden,inter", [(1, 512, 144), (8, 2064, 272), (40, 256, 640),
                                               (130, 400, 208), (600, 272, 528)])
def test_shared_expert(hip, rows, hidden, inter):
    """The chain norm -> gate, up, SwiGLU -> quantisation -> down. The quantised activations are
    compared by their own codes' step: a code may differ by one where the exponential's error
    decides it, which moves an output by at most one scale times one weight value."""
    rng = np.random.default_rng(rows)
    w, d = _expert(rng, inter, hidden)
    xb = wl.bf16_normal(rng, (rows, hidden))
    g = wl._to_bf16_bits((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32))
    mlp = hip.SharedExpertInt8(*d, rows + 3)
    q, s = torch.empty((rows, hidden), dtype=I8, device="cuda"), torch.empty(rows, device="cuda")
    hip.moe_rmsnorm_int8(bf16_dev(xb), bf16_dev(g), q, s)
    out = mlp(q, s, 7.0)
    assert tuple(out.shape) == (rows, hidden)
    qa, sa = q.cpu().numpy(), s.cpu().numpy()
    act = ffn.int8_swiglu(qa, sa, *w[0], *w[1], 7.0)
    s2 = np.max(np.abs(act), axis=1) / 127
    ties = np.abs(np.abs(act / s2[:, None]) % 1 - 0.5) < 127 * 2.0 ** -16  # codes that may flip
    q2 = np.rint(act / s2[:, None])
    ref = (q2 @ w[2][0].astype(np.float64).T) * s2[:, None] * w[2][1]
    flips = (ties.astype(np.float64) @ np.abs(w[2][0]).astype(np.float64).T) * s2[:, None] * w[2][1]
    bound = np.abs(ref) * (2.0 ** -8 + 2.0 ** -16) + flips
    assert np.all(np.abs(f64(out) - ref) <= bound)
    assert np.linalg.norm(flips) < 0.05 * np.linalg.norm(ref)  # the bound says something
    # on BF16 rows, quantised first
    q1, s1 = torch.empty_like(q), torch.empty_like(s)
    x = bf16_dev(xb)
    hip.moe_quant_int8(x, q1, s1)
    want = mlp(q1, s1, 7.0).clone()
    assert torch.equal(mlp.for_combine(x, 7.0), want)


def test_every_row_alone_gives_its_bits(hip):
    """Sums are exact, so a row's outputs are the same in every batch, through every kernel."""
    rng = np.random.default_rng(3)
    m, n, k = 700, 272, 528
    a, w, u = (dev(_codes(rng, r, k)) for r in (m, n, n))
    sa, sw = dev(_scales(rng, m)), dev(_scales(rng, n))
    full = torch.empty((m, n), dtype=BF16, device="cuda")
    act = torch.empty_like(full)
    hip.moe_dense_gemm_int8(a, sa, w, sw, full)
    hip.moe_dense_gate_up_swiglu_int8(a, sa, w, sw, u, sw, act, 7.0)
    for lo, hi in ((0, 1), (3, 19), (100, 140), (100, 164), (200, 500)):
        c = torch.empty((hi - lo, n), dtype=BF16, device="cuda")
        hip.moe_dense_gemm_int8(a[lo:hi], sa[lo:hi], w, sw, c)
        assert torch.equal(c, full[lo:hi])
        hip.moe_dense_gate_up_swiglu_int8(a[lo:hi], sa[lo:hi], w, sw, u, sw, c, 7.0)
        assert torch.equal(c, act[lo:hi])


@pytest.mark.parametrize("m", [3, 50, 200, 800])
def test_captured_and_replayed_on_another_stream(hip, m):
    rng = np.random.default_rng(m)
    w, d = _expert(rng, 144, 256)
    mlp, eager = hip.SharedExpertInt8(*d, m), hip.SharedExpertInt8(*d, m)
    q, s = dev(_codes(rng, m, 256)), dev(_scales(rng, m))
    mlp(q, s, 7.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mlp(q, s, 7.0, stream=side)
    side.synchronize()
    assert torch.equal(got, eager(q, s, 7.0))
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    mlp(q, s, 7.0)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mlp(q, s, 7.0)
    for _ in range(3):
        q.copy_(dev(_codes(rng, m, 256)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager(q, s, 7.0))
        torch.cuda.synchronize()


def test_as_the_shared_term_of_a_layer(hip):
    """moe_layer, moe_layer_decode and moe_layer_few with a SharedExpertInt8: the term it returns."""
    rng = np.random.default_rng(8)
    e, top_k, hidden, mi, rows = 6, 2, 512, 256, 5
    gu = [tuple(dev(t) for t in wl.random_nvfp4(rng, 2 * mi, hidden)) for _ in range(e)]
    dn = [tuple(dev(t) for t in wl.random_nvfp4(rng, hidden, mi)) for _ in range(e)]
    gt = hip.ExpertTable(*zip(*gu), np.full(e, 0.004, np.float32), 2 * mi, hidden)
    dt = hip.ExpertTable(*zip(*dn), np.full(e, 0.01, np.float32), hidden, mi)
    _, d = _expert(rng, 144, hidden)
    mlp = hip.SharedExpertInt8(*d, rows)
    x = bf16_dev(wl.bf16_normal(rng, (rows, hidden)))
    ids = dev(np.array([[0, 1], [2, 0], [5, 3], [1, 4], [2, 3]], np.int32))
    wts = dev(rng.random((rows, top_k)).astype(np.float32))
    term = mlp.for_combine(x, 7.0).clone()
    ws, wd = hip.Workspace(rows, top_k, e, hidden, mi), hip.DecodeWorkspace(rows, top_k, hidden, mi)
    wf = hip.FewWorkspace(rows, top_k, mi)
    for call in (lambda sh, o: hip.moe_layer(x, ids, wts, gt, dt, mi, 7.0, ws, o, sh),
                 lambda sh, o: hip.moe_layer_decode(x, ids, wts, gt, dt, mi, 7.0, wd, o, sh),
                 lambda sh, o: hip.moe_layer_few(x, ids, wts, gt, dt, 7.0, wf, o, sh)):
        a, b, c = (torch.empty_like(x) for _ in range(3))
        call(mlp, a)
        call(term, b)
        call(None, c)
        assert torch.equal(a, b) and not torch.equal(a, c)

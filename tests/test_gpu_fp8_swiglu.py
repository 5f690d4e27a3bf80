"""The SwiGLU forms of the FP8 products on sums that the clamp leaves alone, held to the FP32
form's own bounds by fp8_check (whose CPU tests show what it rejects)."""

import numpy as np
import pytest
import torch

import fp8_check
from oracle import fp8
from test_gpu_fp8 import (POISON8, _counts, _dev, _f8, _host8, _offsets, _out8, _outs, _rest_is,
                          _table)

pytestmark = pytest.mark.gpu

LIMIT = 7.0


def _make(exact):
    return fp8_check.exact_operand if exact else fp8_check.normal_operand


def run_dense(hip, m, n, k, exact):
    """One call against the reference; a second one without the call's own workspace (the form
    in one launch) against it too, with the same bits where the sums are exact."""
    make, rng = _make(exact), np.random.default_rng(m + 5 * n + 11 * k)
    a, sa = make(rng, m, k, False)
    gate, up = make(rng, n, k, True), make(rng, n, k, True)
    want = fp8_check.expected(a, sa, gate, up, LIMIT, exact)
    if m * n > 256:
        assert want.plain > 0.7
    ad, sad, w = _f8(a), _dev(sa), [_f8(gate[0]), _dev(gate[1]), _f8(up[0]), _dev(up[1])]
    qb, q = _out8(m, n)
    sb, s = _outs(m, n)
    hip.moe_dense_gate_up_swiglu_fp8(ad, sad, *w, q, s, LIMIT)
    codes, scale = _host8(q), s.cpu().numpy()
    fp8_check.check(codes, scale, want)
    assert _rest_is(qb, POISON8, m, n) and _rest_is(sb, -7.0, m, fp8.blocks(n))
    if hip.moe_fp8_swiglu_workspace_bytes(m, 0, n, k) == 0:
        return
    q.view(torch.uint8).fill_(POISON8)
    hip._check("one launch", hip.load().moe_dense_gate_up_swiglu_fp8(
        ad.data_ptr(), k, sad.data_ptr(), sad.stride(0), *(t.data_ptr() for t in w), k,
        q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0), m, n, k, LIMIT, None, 0,
        hip._stream(None)))
    fp8_check.check(_host8(q), s.cpu().numpy(), want)
    if exact:
        assert np.array_equal(_host8(q), codes) and np.array_equal(s.cpu().numpy(), scale)


def run_grouped(hip, experts, rows, mi, k, kind, exact, off=None):
    make, rng = _make(exact), np.random.default_rng(experts + 3 * rows + mi + k)
    off = _offsets(_counts(rng, experts, rows, kind)) if off is None else off
    tokens = max(rows // 2, 1)
    a, sa = make(rng, tokens, k, False)
    idx = rng.integers(0, tokens, rows).astype(np.int32)
    pool = [(make(rng, mi, k, True), make(rng, mi, k, True)) for _ in range(min(experts, 5))]
    weights = [None if (experts > 3 and e % 7 == 3) else pool[e % len(pool)]
               for e in range(experts)]
    fused = [None if w is None else tuple(np.concatenate(t) for t in zip(*w)) for w in weights]
    qb, q = _out8(rows, mi)
    sb, s = _outs(rows, mi)
    hip.moe_w8a8_grouped_gemm_swiglu(_f8(a), _dev(sa), _table(hip, fused, 2 * mi, k, True),
                                     _dev(off), q, s, LIMIT, a_gather=_dev(idx))
    codes, scale, written = _host8(q), s.cpu().numpy(), np.zeros(rows, bool)
    # every token's products with every weight of the pool, once
    want = [fp8_check.expected(a, sa, *w, LIMIT, exact) for w in pool]
    for e, lo, hi in fp8.segments(off, rows):
        if weights[e] is None:
            continue
        written[lo:hi] = True
        fp8_check.check(codes[lo:hi], scale[lo:hi], want[e % len(pool)].rows(idx[lo:hi]))
    assert _rest_is(qb, POISON8, rows, mi, written)
    assert _rest_is(sb, -7.0, rows, fp8.blocks(mi), written)


# Sizes of one launch, on every tile; the last ones as large as the workloads' widths.
DENSE = [(1, 16, 16), (1, 144, 272), (40, 272, 656), (77, 1360, 1040), (300, 528, 400),
         (1, 2048, 1040), (46, 144, 1312), (2900, 272, 400), (4300, 400, 272), (3100, 1296, 400)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense(hip, m, n, k, exact):
    run_dense(hip, m, n, k, exact)


GROUPED = [(1, 1, 16, 16, "even"), (8, 6, 128, 272, "even"), (9, 99, 272, 656, "skew"),
           (16, 260, 144, 512, "even"), (16, 1200, 400, 272, "skew"), (20, 3804, 144, 400, "skew"),
           (20, 4890, 400, 400, "skew"), (17, 2400, 784, 400, "even"),
           (70, 9000, 272, 272, "even")]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("experts,rows,mi,k,kind", GROUPED)
def test_grouped(hip, experts, rows, mi, k, kind, exact):
    run_grouped(hip, experts, rows, mi, k, kind, exact)


# Sizes that split K, with the tile and the number of splits each takes (the launcher's rule on
# 256 CUs, pinned on the CPU). Where ways - 1 splits already hold every block of 128 k (25 and 49
# blocks in 8 parts), the last one is empty.
DENSE_SPLIT = [  # tile, ways, m, n, k
    (0, 2, 1034, 144, 1696), (0, 4, 1, 144, 1424), (0, 8, 1, 2048, 6144), (0, 8, 1, 144, 3088),
    (0, 8, 8, 272, 2960), (1, 2, 2053, 144, 3664), (1, 4, 13, 144, 2576), (1, 4, 256, 2048, 6144),
    (1, 8, 13, 144, 5392), (1, 8, 1, 144, 6160), (2, 4, 64, 4144, 2016), (2, 4, 1043, 592, 5984),
    (2, 8, 64, 2080, 3760), (2, 8, 1038, 144, 5856), (2, 8, 64, 2064, 4128),
    (3, 2, 8314, 144, 3984), (3, 4, 99, 4944, 5840), (3, 4, 65, 2704, 1712), (3, 8, 66, 1344, 3024),
    (3, 8, 2063, 144, 5664), (3, 8, 65, 1312, 3088)]
GROUPED_SPLIT = [  # tile, ways, experts, rows, mi, k, counts
    (0, 2, 33, 1041, 144, 1936, "skew"), (0, 4, 3, 6, 144, 1472, "even"),
    (0, 8, 3, 6, 160, 3056, "skew"), (0, 8, 3, 6, 144, 3088, "even"),
    (1, 2, 37, 74, 144, 1792, "skew"), (1, 2, 80, 16, 656, 2960, "even"),
    (1, 4, 3, 39, 160, 2592, "skew"), (1, 8, 3, 45, 144, 5760, "even"),
    (1, 8, 3, 7, 144, 6208, "skew"), (2, 2, 34, 2176, 384, 6096, "even"),
    (2, 4, 3, 192, 2016, 2448, "even"), (2, 8, 3, 192, 1024, 5776, "skew"),
    (3, 2, 35, 1606, 144, 2656, "even"), (3, 4, 21, 972, 192, 3472, "skew"),
    (3, 8, 11, 524, 144, 3056, "skew"), (3, 8, 9, 426, 144, 3152, "even")]


def _ways(hip, experts, rows, n, k):
    return hip.moe_fp8_swiglu_workspace_bytes(rows, experts, n, k) // (rows * n * 8)


@pytest.mark.parametrize("tile,ways,m,n,k", DENSE_SPLIT)
def test_dense_split(hip, tile, ways, m, n, k):
    assert _ways(hip, 0, m, n, k) == ways
    run_dense(hip, m, n, k, True)
    if m * n * k < 3e8:
        run_dense(hip, m, n, k, False)


@pytest.mark.parametrize("tile,ways,experts,rows,mi,k,kind", GROUPED_SPLIT)
def test_grouped_split(hip, tile, ways, experts, rows, mi, k, kind):
    assert _ways(hip, experts, rows, mi, k) == ways
    run_grouped(hip, experts, rows, mi, k, kind, True)
    if rows * mi * k < 3e8:
        run_grouped(hip, experts, rows, mi, k, kind, False)


def test_grouped_split_leaves_uncovered_rows(hip):
    """Rows before the first expert, of absent experts and behind the last one, on each tile."""
    for tile, ways, experts, rows, mi, k, kind in GROUPED_SPLIT:
        if rows * mi * k > 3e8 or rows < 30 or experts <= 3:
            continue
        off = _offsets(_counts(np.random.default_rng(rows), experts, rows - 9, kind)) + 4
        run_grouped(hip, experts, rows, mi, k, kind, True, off)

"""moe_layer_few against the FP64 oracle.

Bounds (``_bounds``), u = 2^-24. Products are exact in FP32 (11 x 8 and 11 x 11 significant bits); a
sum of K of them is off by at most (K + 16) u of the sum of their magnitudes, whatever its order,
and the FP16 rows by 2^-39 of the row's largest value per term below 2^-28 of it. Gate and up take
one rounding by scale2 more. The SwiGLU moves by at most 1.1 L per unit of the gate and by |silu|
per unit of up; its own error is (|g| + 8) u <= 2^-17, its store 2^-11 in FP16 (or half of the
smallest step at a scale of limit^2) and 2^-8 in BF16 (limits over 128). The output adds 2^-8 and
the sums over slots and waves 64 u of the magnitudes.
"""

import numpy as np
import pytest
import torch

import workloads as wl
from gpu_util import bf16_dev, dev, f64
from oracle import codecs, ffn, moe

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U = 2.0 ** -24


class Layer:
    """A small layer: host weights, device tables, scale2."""

    def __init__(self, hip, e, hidden, mi, seed, absent=(), mean=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.e, self.hidden, self.mi = rng, e, hidden, mi
        self.gu = [None if i in absent else wl.random_nvfp4(rng, 2 * mi, hidden) for i in range(e)]
        self.dn = [None if i in absent else wl.random_nvfp4(rng, hidden, mi) for i in range(e)]
        self.s1 = (mean * (0.5 + rng.random(e)) / (6 * np.sqrt(hidden))).astype(np.float32)
        self.s2 = ((0.5 + rng.random(e)) / (6 * np.sqrt(mi))).astype(np.float32)
        self.tables(hip)

    def tables(self, hip):
        def table(ws, s, n, k):
            parts = [(None, None) if w is None else (dev(w[0]), dev(w[1])) for w in ws]
            return hip.ExpertTable(*zip(*parts), s, n, k, device="cuda")
        self.gt = table(self.gu, self.s1, 2 * self.mi, self.hidden)
        self.dt = table(self.dn, self.s2, self.hidden, self.mi)

    def inputs(self, rows, top_k):
        rng = self.rng
        x = wl.bf16_normal(rng, (rows, self.hidden))
        ids = np.stack([rng.permutation(self.e)[:top_k] for _ in range(rows)]).astype(np.int32)
        w = rng.random((rows, top_k)).astype(np.float32)
        return x, ids, w

    def oracle(self, x_bits, ids, w, limit=7.0, shared=None):
        return ffn.few_layer(codecs.bf16_bits_to_f64(x_bits), ids, w, self.gu, self.dn, self.s1,
                             self.s2, limit, shared)


def _bounds(ref, terms, hidden, limit):
    """(per element, of the 2-norm per row) error bounds."""
    mi = terms[0]["act"].size if terms else 0
    elem = np.abs(ref) * 2.0 ** -8 + 1e-30
    norm = np.linalg.norm(ref, axis=1) * 2.0 ** -8 + 1e-30
    lim = min(limit, 1e30)
    for t in terms:
        d = t["mag"] * (hidden + 17) * U * 1.01
        dg, du = d[:mi], d[mi:]
        u_c = np.clip(t["up"], -lim, lim)
        silu = np.abs(t["act"]) / np.maximum(np.abs(u_c), 1e-30)
        store = (2.0 ** -11 if limit <= 128 else 2.0 ** -8) * np.abs(t["act"])
        if limit <= 128:
            store = np.maximum(store, limit * limit * 2.0 ** -38)
        # the clamps cut what gate and up move by
        d_act = 1.1 * np.minimum(dg, 2 * lim) * np.abs(u_c) + (silu + dg) * np.minimum(du, 2 * lim)
        d_act = d_act + store + np.abs(t["act"]) * 2.0 ** -17
        w = np.abs(t["down"])
        sums = (mi + 64) * U * (w @ np.abs(t["act"]))
        elem[t["row"]] += abs(t["p"]) * (w @ d_act + sums)
        spectral = np.linalg.norm(t["down"], 2)
        norm[t["row"]] += abs(t["p"]) * (spectral * np.linalg.norm(d_act) + np.linalg.norm(sums))
    return elem, norm


def _check(got, ref, terms, hidden, limit=7.0):
    elem, norm = _bounds(ref, terms, hidden, limit)
    err = np.abs(got - ref)
    assert np.all(err <= elem), float(np.max(err / elem))
    rows = np.linalg.norm(got - ref, axis=1)
    assert np.all(rows <= norm), float(np.max(rows / norm))


def _run(hip, layer, x, ids, w, limit=7.0, shared=None, ws=None, **kw):
    out = torch.full((x.shape[0], layer.hidden), 9.0, dtype=BF16, device="cuda")
    ws = ws or hip.FewWorkspace(x.shape[0], ids.shape[1], layer.mi)
    hip.moe_layer_few(x, dev(ids), dev(w), layer.gt, layer.dt, limit, ws, out, shared, **kw)
    return out


# hidden: 1, 2, 3 and 4 steps per wave, 1 to 8 waves per item, rows that end inside a step
SIZES = [(1, 4, 64, 64, 2), (2, 5, 256, 192, 3), (3, 8, 512, 320, 4), (5, 6, 768, 256, 2),
         (8, 16, 1088, 448, 4), (4, 3, 2048, 1088, 2), (16, 24, 512, 576, 8), (9, 4, 1536, 256, 1),
         (1, 9, 6144, 2048, 3), (2, 2, 8192, 128, 2), (7, 40, 256, 1280, 6)]


@pytest.mark.parametrize("rows,e,hidden,mi,top_k", SIZES)
def test_layer(hip, rows, e, hidden, mi, top_k):
    layer = Layer(hip, e, hidden, mi, rows * 1000 + hidden)
    x, ids, w = layer.inputs(rows, top_k)
    sh = wl.bf16_normal(layer.rng, (rows, hidden))
    for shared in (None, sh):
        ref, terms = layer.oracle(x, ids, w, shared=None if shared is None else
                                  codecs.bf16_bits_to_f64(shared))
        got = _run(hip, layer, bf16_dev(x), ids, w,
                   shared=None if shared is None else bf16_dev(shared))
        _check(f64(got), ref, terms, hidden)


@pytest.mark.parametrize("rows,top_k,e", [(3, 4, 8), (8, 8, 8), (16, 8, 8), (16, 16, 20), (1, 64, 64),
                                          (1, 200, 256), (2, 128, 300), (12, 8, 2), (16, 5, 7),
                                          (16, 8, 600), (9, 20, 513), (2, 40, 512)])
def test_many_rows_per_expert_and_many_slots(hip, rows, top_k, e):
    """Every number of rows an expert can have, entries swept more than once, over 64 slots."""
    layer = Layer(hip, e, 256, 128, rows + top_k)
    x, ids, w = layer.inputs(rows, min(top_k, e))
    if ids.shape[1] < top_k:
        pad = np.full((rows, top_k - ids.shape[1]), -1, np.int32)
        ids, w = np.hstack([ids, pad]), np.hstack([w, np.ones(pad.shape, np.float32)])
    ref, terms = layer.oracle(x, ids, w)
    _check(f64(_run(hip, layer, bf16_dev(x), ids, w)), ref, terms, 256)


def test_ids_out_of_range_repeated_and_absent(hip):
    layer = Layer(hip, 6, 320, 192, 4, absent=(2, 5))
    for rows in (5, 13):
        x, _, w = layer.inputs(rows, 6)
        ids = layer.rng.integers(-3, 9, (rows, 6)).astype(np.int32)
        ids[0], ids[1], ids[2, :] = -1, 2, 3  # nothing; absent only; the same six times
        ids[3] = [2 ** 31 - 1, -2 ** 31, 6, 0, 1, 0]
        ref, terms = layer.oracle(x, ids, w)
        got = f64(_run(hip, layer, bf16_dev(x), ids, w))
        assert not got[0].any() and not got[1].any()
        _check(got, ref, terms, 320)
        sh = wl.bf16_normal(layer.rng, (rows, 320))
        got = _run(hip, layer, bf16_dev(x), ids, w, shared=bf16_dev(sh))
        assert np.array_equal(f64(got)[:2], codecs.bf16_bits_to_f64(sh)[:2])
    none = Layer(hip, 3, 256, 64, 1, absent=(0, 1, 2))
    x, ids, w = none.inputs(2, 2)
    assert not f64(_run(hip, none, bf16_dev(x), ids, w)).any()


@pytest.mark.parametrize("limit", [0.25, 127.0, 129.0, 1e4, float("inf")])
@pytest.mark.parametrize("rows,e", [(3, 12), (9, 3)])
def test_limits(hip, limit, rows, e):
    """Activations in FP16 up to a limit of 128, in BF16 above; values far past and far within."""
    layer = Layer(hip, e, 512, 448, 6, mean=30.0)
    x, ids, w = layer.inputs(rows, 3)
    ref, terms = layer.oracle(x, ids, w, limit)
    _check(f64(_run(hip, layer, bf16_dev(x), ids, w, limit)), ref, terms, 512, limit)


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -40, 2.0 ** 60])
def test_magnitudes_of_rows(hip, scale):
    """Rows of very different sizes in one batch; each is brought to FP16 by its own power of two.
    scale2 undoes the size, so that the layer's values are ordinary ones."""
    layer = Layer(hip, 5, 512, 256, 7)
    x, ids, w = layer.inputs(4, 2)
    v = codecs.bf16_bits_to_f64(x)
    v[1] *= scale
    v[2] = 0.0
    x = wl._to_bf16_bits(v.astype(np.float32))
    ref, terms = layer.oracle(x, ids, w)
    _check(f64(_run(hip, layer, bf16_dev(x), ids, w)), ref, terms, 512)


@pytest.mark.parametrize("limit", [7.0, 1e4])
def test_what_is_not_finite_stays_in_its_rows(hip, limit):
    layer = Layer(hip, 8, 512, 256, 11)
    x, _, w = layer.inputs(5, 2)
    ids = np.array([[0, 1], [2, 3], [4, 5], [6, 0], [2, 7]], np.int32)
    clean = _run(hip, layer, bf16_dev(x), ids, w, limit).clone()
    xd = bf16_dev(x)
    xd[1, 7] = float("nan")
    got = _run(hip, layer, xd, ids, w, limit)
    assert bool(got[1].isnan().all())
    assert torch.equal(got[[0, 2, 3, 4]], clean[[0, 2, 3, 4]])
    # a NaN block scale of expert 4 (row 2's alone), in either table
    for ws in (layer.gu, layer.dn):
        packed, scales = ws[4]
        bad = scales.copy()
        bad[3, 1] = 0x7F
        ws[4] = (packed, bad)
        layer.tables(hip)
        got = _run(hip, layer, bf16_dev(x), ids, w, limit)
        assert bool(got[2].isnan().any())
        assert torch.equal(got[[0, 1, 3, 4]], clean[[0, 1, 3, 4]])
        ws[4] = (packed, scales)


@pytest.mark.parametrize("rows,e,top_k,hidden", [(1, 256, 8, 512), (5, 64, 6, 320), (16, 300, 8, 256),
                                                 (8, 512, 4, 256), (3, 700, 8, 256), (2, 3, 5, 256),
                                                 (2, 9, 64, 256)])
@pytest.mark.parametrize("kind", ["plain", "bias", "sums", "ties"])
def test_from_logits(hip, rows, e, top_k, hidden, kind):
    """The routing inside the first kernel is moe_router_topk's, ids and weights; the layer is that
    of the given routing."""
    layer = Layer(hip, min(e, 12), hidden, 64, e)
    pick = np.random.default_rng(e).integers(0, layer.e, e)
    layer.gu, layer.dn = [layer.gu[i] for i in pick], [layer.dn[i] for i in pick]
    layer.s1, layer.s2, layer.e = layer.s1[pick], layer.s2[pick], e
    layer.tables(hip)
    rng = layer.rng
    logits = rng.standard_normal((rows, e)).astype(np.float32)
    if kind == "ties":
        logits = np.round(logits)
        logits[:, ::5] = -0.0
    bias = dev(rng.random(e).astype(np.float32)) if kind == "bias" else None
    renorm, scale = kind != "sums", 2.5 if kind == "sums" else 1.0
    wide = torch.full((rows, e + 3), 50.0, device="cuda")
    wide[:, :e] = dev(logits)
    lg = wide[:, :e]
    x = bf16_dev(wl.bf16_normal(rng, (rows, hidden)))
    want_ids = torch.empty((rows, top_k), dtype=torch.int32, device="cuda")
    want_w = torch.empty((rows, top_k), device="cuda")
    hip.moe_router_topk(lg, top_k, want_ids, want_w, bias, scale, renorm)
    ids, w = torch.empty_like(want_ids), torch.empty_like(want_w)
    out, ref = torch.empty_like(x), torch.empty_like(x)
    ws = hip.FewWorkspace(rows, top_k, 64)
    hip.moe_layer_few_from_logits(x, lg, top_k, layer.gt, layer.dt, 7.0, ws, out, bias, scale,
                                  renorm, topk_ids=ids, topk_weights=w)
    assert torch.equal(ids, want_ids)
    if kind == "sums":  # the softmax's sum, by the same tree
        assert torch.allclose(w, want_w, rtol=2.0 ** -20, atol=0)
    else:
        assert torch.equal(w, want_w)
    hip.moe_layer_few(x, ids, w, layer.gt, layer.dt, 7.0, ws, ref)
    assert torch.equal(out, ref)
    again = torch.empty_like(x)
    hip.moe_layer_few_from_logits(x, lg, top_k, layer.gt, layer.dt, 7.0, ws, again, bias, scale,
                                  renorm)
    assert torch.equal(again, out)


def test_near_the_decode_path(hip):
    """The chain of four calls on the same inputs: the same layer but for its BF16 buffers."""
    layer = Layer(hip, 16, 512, 256, 21)
    x, ids, w = layer.inputs(6, 4)
    xd, out = bf16_dev(x), torch.empty((6, 512), dtype=BF16, device="cuda")
    wd = hip.DecodeWorkspace(6, 4, 512, 256)
    hip.moe_layer_decode(xd, dev(ids), dev(w), layer.gt, layer.dt, 256, 7.0, wd, out)
    got = _run(hip, layer, xd, ids, w)
    # weights, gate and up, activations, expert outputs, outputs: 2^-8 each, six together
    assert torch.linalg.norm(got.float() - out.float()) <= 6 * 2.0 ** -8 * torch.linalg.norm(out.float())


def test_strided_rows_and_out_in_place_of_shared(hip):
    layer = Layer(hip, 6, 576, 192, 31)
    x, ids, w = layer.inputs(4, 3)
    sh = wl.bf16_normal(layer.rng, (4, 576))
    want = _run(hip, layer, bf16_dev(x), ids, w, shared=bf16_dev(sh))
    xs = torch.full((4, 600), 1e30, dtype=BF16, device="cuda")
    xs[:, :576] = bf16_dev(x)
    os_ = torch.full((4, 580), 3.0, dtype=BF16, device="cuda")
    os_[:, :576] = bf16_dev(sh)
    ws = hip.FewWorkspace(16, 3, 192)
    view = os_[:, :576]
    hip.moe_layer_few(xs[:, :576], dev(ids), dev(w), layer.gt, layer.dt, 7.0, ws, view, view)
    assert torch.equal(view, want) and bool((os_[:, 576:] == 3.0).all())
    for r in range(4):  # one row, of any stride
        one = torch.empty((1, 576), dtype=BF16, device="cuda")
        hip.moe_layer_few(xs[r:r + 1, :576], dev(ids[r:r + 1]), dev(w[r:r + 1]), layer.gt, layer.dt,
                          7.0, ws, one, bf16_dev(sh[r:r + 1]))
        # sums in another order: each side's own output rounding
        assert torch.linalg.norm(one.float() - want[r].float()) <= 2.0 ** -7 * torch.linalg.norm(
            want[r].float())


def test_no_rows(hip):
    layer = Layer(hip, 3, 256, 64, 2)
    x = torch.empty((0, 256), dtype=BF16, device="cuda")
    ids, w = torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda")
    hip.moe_layer_few(x, ids, w, layer.gt, layer.dt, 7.0, hip.FewWorkspace(1, 2, 64), x.clone())
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,e", [(2, 10), (11, 20)])
def test_captured_replayed_and_on_two_streams(hip, rows, e):
    """A graph through its own workspace, replayed on other inputs beside eager calls; two calls at
    once on two streams; the same bits every time."""
    layer = Layer(hip, e, 512, 320, 41)
    x, _, _ = layer.inputs(rows, 4)
    xd, lg = bf16_dev(x), torch.randn(rows, e, device="cuda")
    ws, ws2 = (hip.FewWorkspace(rows, 4, 320) for _ in range(2))
    out, eager = torch.empty_like(xd), torch.empty_like(xd)

    def call(o, work, stream=None):
        hip.moe_layer_few_from_logits(xd, lg, 4, layer.gt, layer.dt, 7.0, work, o, stream=stream)

    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for _ in range(4):
        xd.copy_(torch.randn(rows, 512, device="cuda").to(BF16))
        lg.copy_(torch.randn(rows, e, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        call(eager, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and bool(eager.any())
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(xd), torch.empty_like(xd)
    torch.cuda.synchronize()
    for _ in range(5):
        call(oa, ws, a)
        call(ob, ws2, b)
    torch.cuda.synchronize()
    assert torch.equal(oa, eager) and torch.equal(ob, eager)


@pytest.mark.parametrize("rows,e,top_k", [(16, 24, 8), (13, 600, 5), (7, 40, 9)])
def test_repeated_and_replayed_calls_and_slots_in_another_order(hip, rows, e, top_k):
    """Slots grouped by every path (a wave's ballots, masks, the scan): repeated calls give the same
    bits, in a replayed graph too; slots in another order stay within the bounds."""
    layer = Layer(hip, min(e, 24), 512, 192, rows)
    pick = np.random.default_rng(e).integers(0, layer.e, e)
    layer.gu, layer.dn = [layer.gu[i] for i in pick], [layer.dn[i] for i in pick]
    layer.s1, layer.s2, layer.e = layer.s1[pick], layer.s2[pick], e
    layer.tables(hip)
    x, ids, w = layer.inputs(rows, top_k)
    xd, idd, wd = bf16_dev(x), dev(ids), dev(w)
    ws, out = hip.FewWorkspace(rows, top_k, 192), torch.empty(rows, 512, dtype=BF16, device="cuda")

    def call(o):
        hip.moe_layer_few(xd, idd, wd, layer.gt, layer.dt, 7.0, ws, o)

    call(out)
    first = out.clone()
    ref, terms = layer.oracle(x, ids, w)
    _check(f64(first), ref, terms, 512)
    for _ in range(5):
        call(out)
        assert torch.equal(out, first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    idd.copy_(dev(ids[:, ::-1].copy()))
    wd.copy_(dev(w[:, ::-1].copy()))
    graph.replay()
    torch.cuda.synchronize()
    _check(f64(out), ref, terms, 512)


def test_a_layer_in_the_order_it_is_used(hip):
    """Norm with the residual, router logits, INT8 shared expert, few-token layer: two layers in a
    row through one residual stream, captured, against the same calls with separate pieces."""
    rows, e, hidden, mi, top_k = 4, 8, 512, 192, 2
    layer = Layer(hip, e, hidden, mi, 51)
    rng = np.random.default_rng(1)
    router = torch.randn(hidden, e, device="cuda") / 20
    w = [(dev(rng.integers(-127, 128, s).astype(np.int8)),
          torch.rand(s[0], device="cuda") / (60 * s[1] ** 0.5)) for s in
         ((144, hidden), (144, hidden), (hidden, 144))]
    mlp = hip.SharedExpertInt8(*w[0], *w[1], *w[2], rows)
    g = bf16_dev(wl._to_bf16_bits((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32)))
    x0 = bf16_dev(wl.bf16_normal(rng, (rows, hidden)))
    r0 = bf16_dev(wl.bf16_normal(rng, (rows, hidden)))
    q, s = torch.empty((rows, hidden), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    y, x, res = (torch.empty_like(x0) for _ in range(3))
    ws = hip.FewWorkspace(rows, top_k, mi)

    def layers():
        x.copy_(x0)
        res.copy_(r0)
        for _ in range(2):
            hip.moe_rmsnorm_int8(x, g, q, s, residual=res, h=res, y=y)
            hip.moe_layer_few_from_logits(y, y.float() @ router, top_k, layer.gt, layer.dt, 7.0, ws,
                                          x, shared=mlp(q, s, 7.0))

    def separate():
        xs, rs = x0.clone(), r0.clone()
        ids = torch.empty((rows, top_k), dtype=torch.int32, device="cuda")
        wt, ys = torch.empty((rows, top_k), device="cuda"), torch.empty_like(xs)
        for _ in range(2):
            rs = (xs.float() + rs.float()).to(BF16)
            hip.moe_rmsnorm_bf16(rs, g, ys)
            hip.moe_rmsnorm_int8(rs, g, q, s)
            hip.moe_router_topk(ys.float() @ router, top_k, ids, wt)
            term = mlp(q, s, 7.0).clone()
            hip.moe_layer_few(ys, ids, wt, layer.gt, layer.dt, 7.0, ws, xs, term)
        return xs, rs

    layers()
    want_x, want_r = separate()
    layers()
    assert torch.equal(x, want_x) and torch.equal(res, want_r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers()
    for _ in range(3):
        x0.copy_(torch.randn(rows, hidden, device="cuda").to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        got_x, got_r = x.clone(), res.clone()
        want_x, want_r = separate()
        assert torch.equal(got_x, want_x) and torch.equal(got_r, want_r)

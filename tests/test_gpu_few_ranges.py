"""moe_layer_few at the ends of its ranges, within the tight bounds of few_check."""

import numpy as np
import pytest

from few_check import assert_exact, bounds, signs
from gpu_util import bf16_dev, f64
from oracle import codecs
from test_gpu_few import Layer, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [0.2, 0.12, 0.08, 0.05, 0.03, 1e-3, 1e-12, 1e-30])
@pytest.mark.parametrize("rows,e", [(3, 12), (9, 3)])
def test_small_limits(hip, limit, rows, e):
    """The gate is clamped from above only: gates near silu's least value beside clamped ups make
    activations of 0.278 limit, far above limit^2."""
    layer = Layer(hip, e, 512, 448, 6, mean=2.0)
    _, ids, w = layer.inputs(rows, 3)
    x = signs(layer.rng, rows, 512)
    assert_exact(layer.gu, codecs.bf16_bits_to_f64(x))
    limit = float(np.float32(limit))
    ref, terms = layer.oracle(x, ids, w, limit)
    assert max(np.abs(t["act"]).max() for t in terms) > 0.278 * limit
    got = f64(_run(hip, layer, bf16_dev(x), ids, w, limit))
    elem = bounds(ref, terms, limit)
    assert np.all(np.abs(got - ref) <= elem), float(np.max(np.abs(got - ref) / elem))


def _without_channel(layer, k):
    """The layer with zero gate and up weights for channel k."""
    for packed, _ in layer.gu:
        packed[:, k // 2] &= 0xF0 if k % 2 == 0 else 0x0F


@pytest.mark.parametrize("spread", [2.0 ** 20, 2.0 ** 31, 2.0 ** 36, 2.0 ** 38, 2.0 ** 39, 2.0 ** 44])
@pytest.mark.parametrize("channel", [0, 301])
def test_values_far_below_the_rows_largest(hip, spread, channel):
    """A channel that all weights skip, `spread` times the other values (-1, 0, 1): these stay what they
    are while they are multiples of 2^-38 of it, and become zeros below."""
    layer = Layer(hip, 5, 512, 192, 9, mean=2.0)
    _without_channel(layer, channel)
    layer.tables(hip)
    _, ids, w = layer.inputs(6, 3)
    x = signs(layer.rng, 6, 512)
    x[:, channel] = 0
    clean = _run(hip, layer, bf16_dev(x), ids, w)
    ref, terms = layer.oracle(x, ids, w)
    assert_exact(layer.gu, codecs.bf16_bits_to_f64(x))
    assert np.all(np.abs(f64(clean) - ref) <= bounds(ref, terms, 7.0))
    rows = [1, 3, 4]
    x[rows, channel] = np.float32(spread).view(np.uint32) >> 16
    got = _run(hip, layer, bf16_dev(x), ids, w)
    gone = spread > 2.0 ** 38
    keep = [r for r in range(6) if not gone or r not in rows]
    assert np.array_equal(f64(got)[keep], f64(clean)[keep])
    assert not gone or not np.any(f64(got)[rows])


@pytest.mark.parametrize("spread,step", [(2.0 ** 35, 2.0 ** -3), (2.0 ** 38, 1.0)])
def test_values_below_the_exact_ones_are_cut_as_stated(hip, spread, step):
    """Values of 8 significant bits in [1, 2) below a skipped channel of `spread`: the layer's outputs are
    those of the values cut towards zero to multiples of 2^-38 spread, bit for bit."""
    layer = Layer(hip, 3, 256, 64, 13, mean=2.0)
    _without_channel(layer, 5)
    layer.tables(hip)
    _, ids, w = layer.inputs(4, 2)
    v = layer.rng.choice([-1.0, 1.0], (4, 256)) * (1 + layer.rng.integers(0, 128, (4, 256)) / 128)
    v[:, 5] = spread
    cut = np.trunc(v / step) * step
    assert_exact(layer.gu, cut, step)

    def bits(a):
        return (a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    got = _run(hip, layer, bf16_dev(bits(v)), ids, w)
    want = _run(hip, layer, bf16_dev(bits(cut)), ids, w)
    assert np.array_equal(f64(got), f64(want)) and np.any(f64(got))
    ref, terms = layer.oracle(bits(cut), ids, w)
    assert np.all(np.abs(f64(got) - ref) <= bounds(ref, terms, 7.0))


@pytest.mark.parametrize("table", ["gt", "dt"])
@pytest.mark.parametrize("field", ["packed_ptrs", "scale_ptrs"])
@pytest.mark.parametrize("rows,e,top_k", [(3, 6, 3), (16, 9, 6), (13, 520, 6)])
def test_an_expert_with_a_null_address_in_one_table(hip, table, field, rows, e, top_k):
    """Weights or scales of either projection: the expert's slots add nothing, on every way of
    grouping the slots."""
    layer = Layer(hip, 6, 320, 192, 17)
    pick = np.arange(e) % 6
    layer.gu, layer.dn = [layer.gu[i] for i in pick], [layer.dn[i] for i in pick]
    layer.s1, layer.s2, layer.e = layer.s1[pick], layer.s2[pick], e
    layer.tables(hip)
    _, ids, w = layer.inputs(rows, top_k)
    x = signs(layer.rng, rows, 320)
    ids[:, 1:][ids[:, 1:] == 1] = 3
    ids[:, 0] = 1
    getattr(getattr(layer, table), field)[1] = 0
    layer.gu[1] = layer.dn[1] = None
    ref, terms = layer.oracle(x, ids, w)
    assert_exact(layer.gu, codecs.bf16_bits_to_f64(x))
    got = f64(_run(hip, layer, bf16_dev(x), ids, w))
    assert np.all(np.abs(got - ref) <= bounds(ref, terms, 7.0)) and np.any(got)


@pytest.mark.parametrize("rows,e,hidden,mi,top_k", [
    (1, 3, 6144, 2048, 2), (3, 2, 8192, 256, 2), (8, 4, 2048, 768, 3), (16, 3, 4096, 448, 2),
    (5, 3, 6208, 320, 3), (2, 5, 64, 2112, 4)])
@pytest.mark.parametrize("limit", [7.0, 100.0])
def test_wide_layers_whose_first_sums_are_exact(hip, rows, e, hidden, mi, top_k, limit):
    """Real widths within bounds that a dropped channel or column does not pass
    (test_few_check.py)."""
    layer = Layer(hip, e, hidden, mi, rows + mi, mean=2.0)
    _, ids, w = layer.inputs(rows, top_k)
    x = signs(layer.rng, rows, hidden)
    assert_exact(layer.gu, codecs.bf16_bits_to_f64(x))
    ref, terms = layer.oracle(x, ids, w, limit)
    got = f64(_run(hip, layer, bf16_dev(x), ids, w, limit))
    elem = bounds(ref, terms, limit)
    assert np.all(np.abs(got - ref) <= elem), float(np.max(np.abs(got - ref) / elem))

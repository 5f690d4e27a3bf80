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

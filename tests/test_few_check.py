"""The bounds of few_check tell a right few-token layer from a slightly wrong one, on the CPU at a
large width: mistakes are planted in the oracle's inputs."""

import numpy as np
import pytest

import workloads as wl
from few_check import assert_exact, bounds, signs
from oracle import codecs, ffn

HIDDEN, MI, E = 6144, 512, 2


@pytest.fixture(scope="module")
def layer():
    rng = np.random.default_rng(5)
    gu = [wl.random_nvfp4(rng, 2 * MI, HIDDEN) for _ in range(E)]
    dn = [wl.random_nvfp4(rng, HIDDEN, MI) for _ in range(E)]
    s1 = ((1.0 + rng.random(E)) / (6 * np.sqrt(HIDDEN))).astype(np.float32)
    s2 = ((0.5 + rng.random(E)) / (6 * np.sqrt(MI))).astype(np.float32)
    x = codecs.bf16_bits_to_f64(signs(rng, 1, HIDDEN))
    x[0, 1234] = 1.0
    assert_exact(gu, x)
    args = dict(x=x, topk_ids=np.array([[0, 1]]), topk_weights=np.array([[0.6, 0.4]], np.float32),
                gate_up=gu, down=dn, scale2_gate_up=s1, scale2_down=s2, limit=7.0)
    ref, terms = ffn.few_layer(**args)
    return args, ref, bounds(ref, terms, 7.0)


def _worst(layer, **kw):
    args, ref, elem = layer
    got, _ = ffn.few_layer(**{**args, **kw})
    return np.max(np.abs(codecs.round_bf16(got) - ref) / elem)


def test_the_formula_rounded_to_bf16_passes(layer):
    assert _worst(layer) <= 1.0


def test_a_dropped_channel_of_a_row(layer):
    x = layer[0]["x"].copy()
    x[0, 1234] = 0.0
    assert _worst(layer, x=x) > 1.0


def test_a_row_taken_from_the_next_channel(layer):
    assert _worst(layer, x=np.roll(layer[0]["x"], 1, axis=1)) > 1.0


@pytest.mark.parametrize("which", ["gate", "up"])
def test_a_dropped_block_of_every_gate_or_up_column(layer, which):
    gu = [tuple(t.copy() for t in w) for w in layer[0]["gate_up"]]
    rows = slice(0, MI) if which == "gate" else slice(MI, 2 * MI)
    for packed, _ in gu:
        packed[rows, 8 * 77:8 * 78] = 0
    assert _worst(layer, gate_up=gu) > 1.0


@pytest.mark.parametrize("rank", [0.5, 0.75, 1.0])
def test_a_dropped_column_of_the_activations(layer, rank):
    """A column whose activation is of the median size or above (a smaller one is worth less than
    the stores' roundings)."""
    _, terms = ffn.few_layer(**layer[0])
    act = abs(terms[0]["p"] * terms[0]["act"])
    column = int(np.argsort(act)[int(rank * (MI - 1))])
    dn = [tuple(t.copy() for t in w) for w in layer[0]["down"]]
    for packed, _ in dn:
        packed[:, column // 2] &= 0x0F if column % 2 else 0xF0
    assert _worst(layer, down=dn) > 1.0


@pytest.mark.parametrize("name", ["scale2_gate_up", "scale2_down"])
def test_a_scale_that_is_two_percent_wrong(layer, name):
    assert _worst(layer, **{name: (layer[0][name] * np.float32(1.02)).astype(np.float32)}) > 1.0


def test_a_dropped_slot_and_zeros(layer):
    assert _worst(layer, topk_ids=np.array([[0, -1]])) > 1.0
    assert _worst(layer, topk_ids=np.array([[-1, -1]])) > 1.0

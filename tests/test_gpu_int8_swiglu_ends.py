"""The INT8 SwiGLU at the ends of its exponential: gates down to where silu leaves BF16's normal numbers.

The exponential's argument and the reciprocal are off by (|g| + 8) 2^-24 of the result, |g| <= 87.34, the
BF16 output by 2^-8. Below g = -126 ln 2 = -87.34 the reciprocal of 1 + e^-g is no normal FP32 number and the
result 0: |silu| is at most 87.34 2^-126 < 1.03e-36 there."""

import numpy as np
import pytest
import torch

from gpu_util import dev, f64
from oracle import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 40, 139, 600, 1559])
@pytest.mark.parametrize("limit", [7.0, 200.0])
def test_gates_of_every_size(hip, m, limit):
    n, k = 512, 16
    gates = np.concatenate([np.linspace(-130, -80, 256), np.linspace(-80, 130, 255), [0.0]])
    gates = gates.astype(np.float32)
    ups = np.tile(np.array([1.0, -3.0, 250.0, 2.0 ** -6], np.float32), n // 4)
    a, w = np.zeros((m, k), np.int8), np.zeros((n, k), np.int8)
    a[:, 3] = w[:, 3] = 1
    act = torch.full((m, n), 5.0, dtype=torch.bfloat16, device="cuda")
    hip.moe_dense_gate_up_swiglu_int8(dev(a), dev(np.ones(m, np.float32)), dev(w), dev(gates), dev(w),
                                      dev(ups), act, limit)
    ref = moe.swiglu_clamp(gates, ups, limit)
    u = np.abs(np.clip(ups.astype(np.float64), -limit, limit))
    bound = np.abs(ref) * (2.0 ** -8 + 2.0 ** -17) + 1.03e-36 * u
    got = f64(act)
    assert np.all(np.abs(got - ref) <= bound)
    normal = gates >= -87.33
    assert np.all(np.abs(got - ref)[:, normal] <= (np.abs(ref) * (2.0 ** -8 + 2.0 ** -17))[normal])
    assert not got[:, gates < -87.34].any()

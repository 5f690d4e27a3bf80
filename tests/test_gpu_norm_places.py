"""Norms that store both the residual stream and the normalised rows in place of their two inputs."""

import numpy as np
import pytest
import torch

import workloads as wl
from gpu_util import bf16_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("cols", [1024, 40000])  # held in registers, formed again
def test_h_over_the_residual_and_y_over_x(hip, form, cols):
    rng = np.random.default_rng(cols)
    xb, rb = (wl.bf16_normal(rng, (5, cols)) for _ in range(2))
    g = bf16_dev(wl.bf16_normal(rng, (1, cols)))[0]

    def call(x, r, h, y):
        q = torch.zeros((5, cols), dtype=torch.int8, device="cuda")
        s = torch.zeros((5, -(-cols // 128)), device="cuda")
        if form == "bf16":
            hip.moe_rmsnorm_bf16(x, g, y, residual=r, h=h)
        elif form == "fp8":
            hip.moe_rmsnorm_fp8(x, g, q.view(torch.float8_e4m3fn), s, residual=r, h=h, y=y)
        else:
            hip.moe_rmsnorm_int8(x, g, q, s.view(-1), residual=r, h=h, y=y)
        return [t.clone() for t in (h, y, q, s)]

    x, r = bf16_dev(xb), bf16_dev(rb)
    want = call(x, r, torch.empty_like(x), torch.empty_like(x))
    for a, b in zip(call(x, r, r, x), want):
        assert torch.equal(a, b)
    with pytest.raises(hip.MoeError, match="h and y"):
        hip.moe_rmsnorm_bf16(x, g, x, residual=r, h=x)

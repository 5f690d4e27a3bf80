"""The norm's E4M3 rows through the FP8 layer that they are made for: moe_rmsnorm_fp8, the router on its
BF16 output, moe_layer_fp8 on its codes with a shared expert on the same codes."""

import numpy as np
import pytest
import torch

import workloads as wl
from gpu_util import bf16_dev
from test_gpu_fp8 import _dev, _layer

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def _bits(v):
    return wl._to_bf16_bits(np.asarray(v, np.float32))


@pytest.mark.parametrize("rows,experts,top_k,hidden,mi,absent", [
    (1, 8, 2, 256, 128, ()), (9, 6, 3, 272, 144, (2,)), (70, 12, 3, 384, 272, ())])
def test_codes_in_place_of_rows(hip, rows, experts, top_k, hidden, mi, absent):
    """Rows whose norm is exact in BF16 (mean square 1, powers of two as weights): the norm's codes are the
    quantiser's, so the layer on codes gives the bits of the layer on BF16 rows."""
    rng, _, _, _, (gt, dt), ws, sh = _layer(hip, rows, rows, experts, top_k, hidden, mi, absent, True)
    x = bf16_dev(_bits(rng.choice([-1.0, 1.0], (rows, hidden))))
    g = bf16_dev(_bits(2.0 ** rng.integers(-3, 4, hidden)))
    ids = _dev(np.stack([rng.permutation(experts)[:top_k] for _ in range(rows)]).astype(np.int32))
    w = _dev(rng.random((rows, top_k)).astype(np.float32))
    y, q = torch.empty_like(x), torch.empty((rows, hidden + 16), dtype=F8, device="cuda")
    q, s = q[:, :hidden], torch.empty((rows, -(-hidden // 128)), device="cuda")
    hip.moe_rmsnorm_fp8(x, g, q, s, 0.0, y=y)
    term = bf16_dev(wl.bf16_normal(rng, (rows, hidden)))
    for shared in (None, term, sh):
        want, got = torch.empty_like(x), torch.empty_like(x)
        hip.moe_layer_fp8(y, ids, w, gt, dt, 7.0, ws, want, shared)
        ws.x.view(torch.uint8).fill_(0x7F)  # the layer's own buffers have no part in it
        ws.x_scale.fill_(float("nan"))
        hip.moe_layer_fp8(q, ids, w, gt, dt, 7.0, ws, got, shared, x_scale=s)
        assert torch.equal(got, want) and bool(got.any())


def test_norm_router_and_layer_captured(hip):
    rows, experts, top_k, hidden, mi = 33, 10, 2, 512, 160
    rng, _, _, _, (gt, dt), ws, sh = _layer(hip, 4, rows, experts, top_k, hidden, mi, (3,), True)
    x, res = (bf16_dev(wl.bf16_normal(rng, (rows, hidden))) for _ in range(2))
    g = bf16_dev(_bits(1 + 0.1 * rng.standard_normal(hidden)))
    router = torch.randn(hidden, experts, device="cuda") / 20

    def buffers():
        return dict(h=torch.empty_like(x), y=torch.empty_like(x),
                    q=torch.empty((rows, hidden), dtype=F8, device="cuda"),
                    s=torch.empty((rows, hidden // 128), device="cuda"),
                    ids=torch.empty((rows, top_k), dtype=torch.int32, device="cuda"),
                    w=torch.empty((rows, top_k), device="cuda"), out=torch.empty_like(x))

    def step(b, work):
        hip.moe_rmsnorm_fp8(x, g, b["q"], b["s"], residual=res, h=b["h"], y=b["y"])
        hip.moe_router_topk(b["y"].float() @ router, top_k, b["ids"], b["w"])
        hip.moe_layer_fp8(b["q"], b["ids"], b["w"], gt, dt, 7.0, work, b["out"], sh, x_scale=b["s"])

    a, e = buffers(), buffers()
    step(a, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, ws)
    ws2 = hip.Fp8Workspace(rows, top_k, experts, hidden, mi)
    for _ in range(3):
        x.copy_(torch.randn(rows, hidden, device="cuda").to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = a["out"].clone()
        step(e, ws2)
        torch.cuda.synchronize()
        assert torch.equal(got, e["out"]) and torch.equal(a["h"], e["h"]) and bool(got.any())
        # the codes come from the unrounded norm: a second quantiser would start from BF16
        q = torch.empty_like(e["q"])
        hip.moe_quant_fp8(e["y"], q, torch.empty_like(e["s"]))
        assert not torch.equal(q.view(torch.uint8), e["q"].view(torch.uint8))

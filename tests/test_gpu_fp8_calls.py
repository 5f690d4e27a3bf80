"""Calls of the FP8 operators that the binding has to bring into the library's form."""

import pytest
import torch

pytestmark = pytest.mark.gpu

F8, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.mark.parametrize("gap", [3, 1 << 22])
def test_one_row_of_any_stride(hip, gap):
    """The last row of buffers whose rows are an odd number of values (or over 2^22) apart:
    the bits of the same row on its own."""
    torch.manual_seed(1)
    k, n = 272, 144
    x = torch.randn(1, k, device="cuda").to(BF16)
    w = torch.randint(0, 120, (n, k), dtype=torch.uint8, device="cuda")
    sw = torch.rand(2, 3, device="cuda")

    def row(cols, dtype):
        t = torch.zeros(cols, dtype=dtype, device="cuda").as_strided((1, cols), (cols + gap, 1))
        assert t.stride(0) == cols + gap
        return t

    def chain(new):
        xr, q, s = new(k, BF16), new(k, F8), new(3, torch.float32)
        c, act, act_s = new(n, BF16), new(n, F8), new(2, torch.float32)
        xr.copy_(x)
        hip.moe_quant_fp8(xr, q, s)
        hip.moe_dense_gemm_fp8(q, s, w, sw, c)
        hip.moe_dense_gate_up_swiglu_fp8(q, s, w, sw, w, sw, act, act_s, 7.0)
        return [t.contiguous().clone() for t in (q.view(torch.uint8), s, c, act.view(torch.uint8),
                                                 act_s)]

    plain = chain(lambda cols, dtype: torch.zeros((1, cols), dtype=dtype, device="cuda"))
    for got, want in zip(chain(row), plain):
        assert torch.equal(got, want)


def test_quantising_no_columns(hip):
    for rows in (0, 3):
        hip.moe_quant_fp8(torch.empty((rows, 0), dtype=BF16, device="cuda"),
                          torch.empty((rows, 0), dtype=F8, device="cuda"),
                          torch.empty((rows, 0), device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [1, 8, 60])
def test_a_layer_call_allocates_nothing(hip, rows):
    """Everything a layer with its shared expert needs, the split-K sums among it, lies in the
    workspace objects; every row count up to theirs gives the bits of objects of its own size."""
    torch.manual_seed(rows)
    experts, top_k, hidden, mi, max_rows = 6, 2, 2064, 144, 70
    assert hip.moe_fp8_swiglu_workspace_bytes(rows * top_k, experts, mi, hidden) > 0
    assert hip.moe_fp8_swiglu_workspace_bytes(rows, 0, mi, hidden) > 0

    def weight(n, k):
        w = torch.randint(0, 120, (n, k), dtype=torch.uint8, device="cuda")
        return w, torch.rand(-(-n // 128), -(-k // 128), device="cuda") / 1000

    gu = [tuple(torch.cat(t) for t in zip(weight(mi, hidden), weight(mi, hidden)))
          for _ in range(experts)]
    dn = [weight(hidden, mi) for _ in range(experts)]
    gt = hip.Fp8ExpertTable(*zip(*gu), 2 * mi, hidden, gate_up=True)
    dt = hip.Fp8ExpertTable(*zip(*dn), hidden, mi)
    sh_w = [t for w in (weight(mi, hidden), weight(mi, hidden), weight(hidden, mi)) for t in w]
    x = torch.randn(rows, hidden, device="cuda").to(BF16)
    ids = torch.rand(rows, experts, device="cuda").argsort(1)[:, :top_k].int().contiguous()
    w = torch.rand(rows, top_k, device="cuda")
    outs = []
    for most in (max_rows, rows):
        ws = hip.Fp8Workspace(most, top_k, experts, hidden, mi)
        shared = hip.SharedExpertFp8(*sh_w, most)
        out = torch.empty((rows, hidden), dtype=BF16, device="cuda")
        hip.moe_layer_fp8(x, ids, w, gt, dt, 7.0, ws, out, shared)
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        hip.moe_layer_fp8(x, ids, w, gt, dt, 7.0, ws, out, shared)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("own_workspace", [False, True])
def test_split_products_captured_and_replayed(hip, own_workspace):
    """Split-K SwiGLU calls in a graph, dense and grouped, through the caller's workspace and the
    call's own (from the graph's pool); every replay on other inputs, with eager calls of the
    same sizes between the replays, against the eager result."""
    torch.manual_seed(3)
    m, n, k, experts = 12, 144, 2064, 4
    need = max(hip.moe_fp8_swiglu_workspace_bytes(m, e, n, k) for e in (0, experts))
    assert min(hip.moe_fp8_swiglu_workspace_bytes(m, e, n, k) for e in (0, experts)) > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if own_workspace else None

    def weight(rows, blocks):
        w = torch.randint(0, 120, (rows, k), dtype=torch.uint8, device="cuda")
        return w, torch.rand(blocks, 17, device="cuda") / 1000

    gate, up = weight(n, 2), weight(n, 2)
    table = hip.Fp8ExpertTable(*zip(*[weight(2 * n, 4) for _ in range(experts)]), 2 * n, k,
                               gate_up=True)
    off = torch.tensor([0, 5, 5, 9, 12], dtype=torch.int32, device="cuda")
    a = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    sa = torch.empty((m, 17), device="cuda")

    def outputs():
        return [(torch.zeros((m, n), dtype=torch.uint8, device="cuda"),
                 torch.zeros((m, 2), device="cuda")) for _ in range(2)]

    def calls(out, work):
        hip.moe_dense_gate_up_swiglu_fp8(a, sa, *gate, *up, *out[0], 7.0, workspace=work)
        hip.moe_w8a8_grouped_gemm_swiglu(a, sa, table, off, *out[1], 7.0, workspace=work)

    def fill():
        a.copy_(torch.randint(0, 120, (m, k), dtype=torch.uint8, device="cuda"))
        sa.copy_(torch.rand(m, 17, device="cuda"))

    fill()
    captured, eager = outputs(), outputs()
    calls(captured, ws)  # attributes are set before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(captured, ws)
    for _ in range(4):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        calls(eager, None)
        torch.cuda.synchronize()
        for got, want in zip(captured, eager):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert bool(want[0].any())

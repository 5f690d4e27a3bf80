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

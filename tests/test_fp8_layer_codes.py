"""moe_layer_fp8 on quantised rows, on the host: which arguments it hands on, what it refuses."""

import pytest
import torch

import grouped_nvfp4_w4a16_amd as pkg
from test_fp8_binding import BF16, F8, F32, I32, Table, Tensor, Workspace, lib  # noqa: F401


class Buffer(Tensor):
    def __getitem__(self, rows):
        return Buffer((min(rows.stop, self.shape[0]), *self.shape[1:]), self.dtype)


class Layer(Workspace):
    """Every buffer of an Fp8Workspace for 4 rows."""

    def __init__(self):
        super().__init__()
        self.sorted_token_ids, self.sorted_expert_ids, self.token_to_perm = (
            Buffer((8,), I32) for _ in range(3))
        self.expert_offsets = Buffer((4,), I32)
        self.x, self.x_scale = Buffer((4, 256), F8, ptr=0x20000), Buffer((4, 2), F32, ptr=0x30000)
        self.act, self.act_scale = Buffer((8, 144), F8), Buffer((8, 2), F32)
        self.expert_out = Buffer((8, 256), BF16)
        self.split = Buffer((1024,), torch.uint8)


class Bf16Expert(pkg.SharedExpert):
    def __init__(self):
        self.out = Tensor((4, 256), BF16)


class Int8Expert(pkg.SharedExpertInt8):
    def __init__(self):
        self.out = Tensor((4, 256), BF16)


def _call(x, x_scale=None, shared=None):
    pkg.moe_layer_fp8(x, Tensor((4, 2), I32), Tensor((4, 2), F32), Table(3, 288, 256, True),
                      Table(3, 256, 144), 7.0, Layer(), Tensor((4, 256), BF16), shared,
                      x_scale=x_scale)


CODES, SCALES = Tensor((4, 256), F8, (272, 1), ptr=0x40000), Tensor((4, 2), F32, (3, 1), ptr=0x50000)


def test_codes_go_to_the_product_and_nothing_is_quantised(lib):  # noqa: F811
    _call(CODES, SCALES)
    calls = dict(lib.calls)
    assert [n for n, _ in lib.calls] == ["moe_align", "moe_w8a8_grouped_gemm_swiglu",
                                         "moe_w8a8_grouped_gemm", "moe_combine"]
    product = calls["moe_w8a8_grouped_gemm_swiglu"]
    assert product[0] == 0x40000 and product[1] == 272 and 0x50000 in product and 3 in product
    _call(Tensor((4, 256), BF16))
    assert "moe_quant_fp8" in dict(lib.calls)


@pytest.mark.parametrize("x,scale,error", [
    (Tensor((4, 256), BF16), SCALES, TypeError), (CODES, Tensor((4, 2), BF16), TypeError),
    (CODES, Tensor((4, 1), F32), ValueError), (CODES, Tensor((3, 2), F32), ValueError),
    (CODES, Tensor((4, 2), F32, (4, 2)), ValueError), (Tensor((4, 256), F8, (512, 2)), SCALES, ValueError),
    (Tensor((3, 256), F8), SCALES, ValueError), (Tensor((4, 128), F8), SCALES, ValueError),
    (Tensor((4, 256), F8, device=1), SCALES, ValueError),
    (CODES, Tensor((4, 2), F32, device=1), ValueError)])
def test_what_does_not_fit_launches_nothing(lib, x, scale, error):  # noqa: F811
    with pytest.raises(error):
        _call(x, scale)
    assert lib.calls == []


@pytest.mark.parametrize("expert", [Bf16Expert, Int8Expert])
def test_experts_on_bf16_rows_are_refused_with_codes(lib, expert):  # noqa: F811
    with pytest.raises(ValueError, match="BF16 rows"):
        _call(CODES, SCALES, expert())
    assert lib.calls == []

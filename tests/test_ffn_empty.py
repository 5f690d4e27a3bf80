"""The norm and the row quantiser without rows or columns, on the host: nothing is enqueued, so
nothing is written, and no pointer is asked for."""

import pytest

import grouped_nvfp4_w4a16_amd as pkg
from test_ffn_binding import lib as binding_lib, norm_args  # noqa: F401
from test_ffn_library import N, lib  # noqa: F401


@pytest.mark.parametrize("rows,cols", [(0, 256), (5, 0), (0, 0)])
def test_the_library_enqueues_nothing(lib, rows, cols):  # noqa: F811
    """No pointers at all: a call that enqueued a kernel would need them (and a GPU)."""
    norm = (N, 256, N, 0, N, 1e-6, N, 0, N, 256)
    assert lib.moe_rmsnorm_bf16(*norm, rows, cols, N) == 0
    assert lib.moe_rmsnorm_fp8(*norm, N, 256, N, 2, rows, cols, N) == 0
    assert lib.moe_rmsnorm_int8(*norm, N, 256, N, rows, cols, N) == 0
    assert lib.moe_quant_int8(N, 256, N, 256, N, rows, cols, N) == 0


@pytest.mark.parametrize("name", sorted(norm_args()))
def test_the_binding_calls_nothing_without_columns(binding_lib, name):  # noqa: F811
    getattr(pkg, name)(**norm_args(5, 0)[name])
    assert binding_lib.calls == []

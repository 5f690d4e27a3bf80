"""The INT8 products' largest sizes on the host: what would run past 32 bits is refused by its size,
before anything is launched."""

import ctypes

import pytest

from test_ffn_library import GEMM, N, lib  # noqa: F401

TOP = 2 ** 31 - 256  # the most rows and output columns


def _calls(lib, **kw):
    a = {**GEMM, "lda": 16, "ldb": 16, "k": 16, **kw}
    yield lib.moe_dense_gemm_int8(a["a"], a["lda"], a["sa"], a["b"], a["ldb"], a["sb"], a["c"],
                                  a["ldc"], a["m"], a["n"], a["k"], N)
    yield lib.moe_dense_gate_up_swiglu_int8(
        a["a"], a["lda"], a["sa"], a["b"], a["sb"], a["u"], a["su"], a["ldb"], a["c"], a["ldc"],
        a["m"], a["n"], a["k"], a["limit"], N)


@pytest.mark.parametrize("m,n", [(TOP + 1, 16), (2 ** 31 - 1, 16), (2 ** 31 - 1, 1 << 20),
                                 (0, TOP + 16), (1, TOP + 16), (2 ** 31 - 1, TOP + 16)])
def test_rows_and_columns_past_the_last_whole_tile(lib, m, n):  # noqa: F811
    for status in _calls(lib, m=m, n=n, ldc=n):
        assert status == 1
        assert b"2147483392" in lib.moe_w4a16_last_error()


@pytest.mark.parametrize("m,n", [(TOP, 1 << 20), (1 << 20, TOP), (TOP, TOP)])
def test_more_tiles_than_a_launch_holds(lib, m, n):  # noqa: F811
    for status in _calls(lib, m=m, n=n, ldc=n):
        assert status == 1
        assert b"too large" in lib.moe_w4a16_last_error()


def test_no_rows_of_the_widest_output(lib):  # noqa: F811
    for status in _calls(lib, m=0, n=TOP, ldc=TOP):
        assert status == 0


def test_the_shared_experts_widths(lib):  # noqa: F811
    p = ctypes.c_void_p(0x10000)
    for inter, hidden in ((TOP + 16, 512), (512, TOP + 16)):
        assert lib.moe_shared_expert_int8(p, 512, p, p, p, p, p, 512, p, 512, p, p, hidden, 0, inter,
                                          hidden, 7.0, p, 1 << 40, N) == 1

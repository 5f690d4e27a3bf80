"""The tile rule of the INT8 products, built for the host from the library's own source: its tiles,
and that the GPU tests reach each of them."""

import ctypes
import os
import subprocess

import pytest

import test_gpu_int8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "grouped_nvfp4_w4a16_amd", "csrc")
_SHIM = """
#include "int8_plan.h"
extern "C" int tiles() { return moe::kInt8Tiles; }
extern "C" int built(int swiglu, int t) { return moe::int8_shape(swiglu, t).step != 0; }
extern "C" int rows(int swiglu, int t) { return moe::int8_shape(swiglu, t).rows; }
extern "C" int tile(int swiglu, long m, long n, long k) { return moe::int8_tile(swiglu, m, n, k); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("int8_plan")
    (d / "plan.cpp").write_text(_SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", CSRC,
                    str(d / "plan.cpp"), "-o", str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    lib.tile.argtypes = [ctypes.c_int] + [ctypes.c_long] * 3
    return lib


@pytest.mark.parametrize("swiglu", [0, 1])
def test_the_gpu_tests_reach_every_tile(plan, swiglu):
    built = {t for t in range(plan.tiles()) if plan.built(swiglu, t)}
    assert len(built) == (9 if not swiglu else 7)
    assert {plan.tile(swiglu, m, n, k) for m, n, k in test_gpu_int8.SIZES} == built


@pytest.mark.parametrize("swiglu", [0, 1])
def test_few_rows_take_few_row_tiles_and_many_take_large_ones(plan, swiglu):
    for n, k in ((6144, 2048), (2048, 6144), (144, 2048)):
        assert plan.rows(swiglu, plan.tile(swiglu, 1, n, k)) <= 32
    for m in (1, 17, 300, 1 << 22, (1 << 31) - 1):
        for n, k in ((16, 16), (16, 131056), (1 << 20, 128)):
            assert plan.built(swiglu, plan.tile(swiglu, m, n, k))
    assert plan.rows(swiglu, plan.tile(swiglu, 16384, 6144, 2048)) == 256

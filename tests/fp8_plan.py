"""The tile rule of the FP8 products, built for the host from the library's own source (test
infrastructure only)."""

import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "grouped_nvfp4_w4a16_amd", "csrc", "fp8_plan.h")
CUS = 256

_SHIM = """
#include "fp8_plan.h"
extern "C" void tile(int swiglu, int t, int *rows, int *width) {
  const moe::Fp8Tile s = swiglu ? moe::fp8_tile<true>(t) : moe::fp8_tile<false>(t);
  *rows = s.rows, *width = s.width;
}
extern "C" void plan(int swiglu, long rows, long experts, long n, long k, int split, int cus,
                     int *tile, int *ways) {
  const moe::Fp8Plan p = swiglu ? moe::fp8_plan<true>(rows, experts, n, k, split, cus)
                                : moe::fp8_plan<false>(rows, experts, n, k, split, cus);
  *tile = p.tile, *ways = p.ways;
}
"""


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, out = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(_SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I",
                        os.path.dirname(SOURCE), src, "-o", out], check=True)
        lib = ctypes.CDLL(out)
    lib.plan.argtypes = [ctypes.c_int] + [ctypes.c_long] * 4 + [ctypes.c_int] * 2 + \
        [ctypes.c_void_p] * 2
    lib.tile.argtypes = [ctypes.c_int] * 2 + [ctypes.c_void_p] * 2
    return lib


def plan(swiglu, rows, experts, n, k, split=True):
    """(tile, ways) the launcher takes on 256 CUs; ``split``: with a workspace."""
    t, w = ctypes.c_int(), ctypes.c_int()
    _lib().plan(int(swiglu), rows, experts, n, k, int(split), CUS, ctypes.byref(t), ctypes.byref(w))
    return t.value, w.value


def tile(swiglu, t):
    """(rows, weight rows) of tile t."""
    r, w = ctypes.c_int(), ctypes.c_int()
    _lib().tile(int(swiglu), t, ctypes.byref(r), ctypes.byref(w))
    return r.value, w.value

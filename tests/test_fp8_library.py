"""The FP8 calls' refusals on the host: bad arguments return MOE_EINVAL before anything
reaches the GPU, empty ones return MOE_OK (no launch happens here)."""

import ctypes
import os

import pytest

import grouped_nvfp4_w4a16_amd as pkg
from grouped_nvfp4_w4a16_amd import build as builder

N = None


def _p(v=0x1000):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkg.LIB_PATH):
        builder.build()
    return pkg.load()


def test_quant(lib):
    base = dict(x=_p(), ld_x=256, q=_p(), ld_q=256, s=_p(), ld_s=2, rows=0, cols=256)

    def call(**kw):
        a = {**base, **kw}
        return lib.moe_quant_fp8(a["x"], a["ld_x"], a["q"], a["ld_q"], a["s"], a["ld_s"],
                                 a["rows"], a["cols"], N)
    assert call() == 0
    assert call(rows=4, cols=0) == 0
    for kw in (dict(rows=-1), dict(cols=-16), dict(cols=250), dict(ld_x=248), dict(ld_x=260),
               dict(ld_q=240), dict(ld_q=264), dict(ld_s=1), dict(rows=4, x=N),
               dict(rows=4, q=N), dict(rows=4, s=N), dict(rows=4, x=_p(0x1008)),
               dict(rows=4, q=_p(0x1008)), dict(rows=4, s=_p(0x1002)),
               dict(rows=2 ** 31 - 1, cols=128 * 2 ** 10, ld_x=2 ** 17, ld_q=2 ** 17, ld_s=2 ** 10)):
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"quant_fp8")


def test_dense(lib):
    base = dict(a=_p(), lda=512, sa=_p(), lds=4, b=_p(), ldb=512, sb=_p(), c=_p(), ldc=144, m=0,
                n=144, k=512)

    def call(**kw):
        a = {**base, **kw}
        return lib.moe_dense_gemm_fp8(a["a"], a["lda"], a["sa"], a["lds"], a["b"], a["ldb"],
                                      a["sb"], a["c"], a["ldc"], a["m"], a["n"], a["k"], N)
    assert call() == 0
    for kw in (dict(m=-1), dict(n=0), dict(n=136), dict(k=0), dict(k=500), dict(k=32784, lda=32784,
               ldb=32784, lds=300), dict(lda=496), dict(lda=520), dict(ldb=500), dict(lds=3),
               dict(ldc=128), dict(ldc=148), dict(lda=1 << 22), dict(ldb=1 << 22),
               dict(lds=1 << 20), dict(m=3, a=N), dict(m=3, sa=N), dict(m=3, b=N), dict(m=3, sb=N),
               dict(m=3, c=N), dict(m=3, a=_p(0x1008)), dict(m=3, b=_p(0x1008)),
               dict(m=3, c=_p(0x1008)), dict(m=3, sa=_p(0x1001)), dict(m=3, sb=_p(0x1002))):
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"dense_gemm_fp8")


def test_dense_swiglu(lib):
    base = dict(a=_p(), lda=512, sa=_p(), lds=4, g=_p(), sg=_p(), u=_p(), su=_p(), ldw=512,
                act=_p(), ld_act=272, os=_p(), ld_os=3, m=0, n=272, k=512, limit=7.0, ws=N, wb=0)

    def call(**kw):
        a = {**base, **kw}
        return lib.moe_dense_gate_up_swiglu_fp8(
            a["a"], a["lda"], a["sa"], a["lds"], a["g"], a["sg"], a["u"], a["su"], a["ldw"],
            a["act"], a["ld_act"], a["os"], a["ld_os"], a["m"], a["n"], a["k"], a["limit"],
            a["ws"], a["wb"], N)
    assert call() == 0
    for kw in (dict(limit=0.0), dict(limit=-1.0), dict(limit=float("nan")), dict(ld_act=264),
               dict(ld_act=280), dict(ld_os=2), dict(n=264), dict(m=2, g=N), dict(m=2, u=N),
               dict(m=2, sg=N), dict(m=2, su=N), dict(m=2, act=N), dict(m=2, os=N),
               dict(m=2, act=_p(0x1008)), dict(m=2, u=_p(0x1004)), dict(ldw=500),
               dict(ws=_p(0x1010), wb=1 << 30)):
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"dense_gate_up_swiglu_fp8")


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped(lib, swiglu):
    base = dict(a=_p(), lda=512, sa=_p(), lds=4, a_rows=8, g=N, wp=_p(), sp=_p(), off=_p(), e=4,
                out=_p(), ldo=272, os=_p(), ld_os=3, rows=0, n=272, k=512, limit=7.0, ws=N, wb=0)

    def call(**kw):
        a = {**base, **kw}
        head = (a["a"], a["lda"], a["sa"], a["lds"], a["a_rows"], a["g"], a["wp"], a["sp"],
                a["off"], a["e"], a["out"], a["ldo"])
        if swiglu:
            return lib.moe_w8a8_grouped_gemm_swiglu(*head, a["os"], a["ld_os"], a["rows"], a["n"],
                                                    a["k"], a["limit"], a["ws"], a["wb"], N)
        return lib.moe_w8a8_grouped_gemm(*head, a["rows"], a["n"], a["k"], N)
    assert call() == 0
    for kw in (dict(rows=-1), dict(e=0), dict(e=2049), dict(a_rows=-1), dict(rows=4, a_rows=0),
               dict(rows=9), dict(rows=4, wp=N), dict(rows=4, sp=N), dict(rows=4, off=N),
               dict(rows=4, a=N), dict(rows=4, out=N), dict(n=264), dict(k=520), dict(lds=3),
               dict(rows=4, g=_p(), a_rows=1 << 22, lda=512),
               dict(rows=4, g=_p(), a_rows=1 << 20, lds=1 << 10)):
        assert call(**kw) == 1, kw
        assert b"w8a8_grouped_gemm" in lib.moe_w4a16_last_error()


def test_swiglu_workspace_query(lib):
    for rows, width, k in ((1, 2048, 6144), (256, 2048, 6144), (16, 512, 2048)):
        need = lib.moe_fp8_swiglu_workspace_bytes(rows, 0, width, k)
        ways = need // (rows * width * 8)  # FP32 gate and up sums per split
        assert ways in (2, 4, 8) and need == ways * rows * width * 8
    for args in ((0, 0, 2048, 6144), (-1, 0, 64, 64), (4, -1, 64, 64), (4, 0, 0, 64),
                 (4, 0, 64, 0), (4096, 0, 2048, 6144), (2048, 256, 2048, 6144), (1, 0, 64, 128)):
        assert lib.moe_fp8_swiglu_workspace_bytes(*args) == 0, args

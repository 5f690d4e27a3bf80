"""Refusals on the host of the norm, the INT8 calls and the few-token layer: bad arguments return
MOE_EINVAL (or MOE_ECAPACITY) before anything reaches the GPU, empty ones MOE_OK."""

import ctypes
import os

import pytest

import grouped_nvfp4_w4a16_amd as pkg
from grouped_nvfp4_w4a16_amd import build as builder

N = None
NAN, INF = float("nan"), float("inf")


def _p(v=0x10000):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkg.LIB_PATH):
        builder.build()
    return pkg.load()


@pytest.mark.parametrize("form", ["bf16", "fp8", "int8"])
def test_rmsnorm(lib, form):
    base = dict(x=_p(), ld_x=256, r=_p(), ld_r=256, g=_p(), eps=1e-6, h=_p(), ld_h=256, y=_p(),
                ld_y=256, q=_p(), ld_q=256, s=_p(), ld_s=2, rows=0, cols=256)

    def call(**kw):
        a = {**base, **kw}
        args = [a[n] for n in ("x", "ld_x", "r", "ld_r", "g", "eps", "h", "ld_h", "y", "ld_y")]
        if form != "bf16":
            args += [a["q"], a["ld_q"], a["s"]]
        if form == "fp8":
            args.append(a["ld_s"])
        return getattr(lib, "moe_rmsnorm_" + form)(*args, a["rows"], a["cols"], N)
    assert call() == 0
    assert call(rows=4, cols=0) == 0
    bad = [dict(rows=-1), dict(cols=-8), dict(cols=252), dict(ld_x=248), dict(ld_x=260),
           dict(ld_r=128), dict(ld_r=257), dict(ld_h=255), dict(ld_y=8), dict(eps=-1e-9),
           dict(eps=NAN), dict(eps=INF), dict(rows=4, x=N), dict(rows=4, g=N),
           dict(rows=4, x=_p(0x10008)), dict(rows=4, r=_p(0x10002)), dict(rows=4, g=_p(0x10004)),
           dict(rows=4, h=_p(0x10008)), dict(rows=4, y=_p(0x10008)), dict(rows=1 << 22)]
    if form == "bf16":
        bad.append(dict(rows=4, y=N))
    else:
        bad += [dict(ld_q=248), dict(ld_q=260), dict(rows=4, q=N), dict(rows=4, s=N),
                dict(rows=4, q=_p(0x10004)), dict(rows=4, s=_p(0x10002))]
    if form == "fp8":
        bad.append(dict(ld_s=1))
    for kw in bad:
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"rmsnorm_" + form.encode()), kw


def test_quant_int8(lib):
    base = dict(x=_p(), ld_x=256, q=_p(), ld_q=256, s=_p(), rows=0, cols=256)

    def call(**kw):
        a = {**base, **kw}
        return lib.moe_quant_int8(a["x"], a["ld_x"], a["q"], a["ld_q"], a["s"], a["rows"],
                                  a["cols"], N)
    assert call() == 0 and call(rows=3, cols=0) == 0
    for kw in (dict(rows=-1), dict(cols=100), dict(ld_x=128), dict(ld_q=250), dict(rows=2, x=N),
               dict(rows=2, q=N), dict(rows=2, s=N), dict(rows=2, x=_p(0x10008)),
               dict(rows=1 << 30)):
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"quant_int8"), kw


GEMM_BAD = [dict(m=-1), dict(n=0), dict(n=136), dict(k=0), dict(k=500),
            dict(k=131072, lda=131072, ldb=131072), dict(lda=496), dict(lda=520), dict(ldb=500),
            dict(ldb=504), dict(ldc=128), dict(ldc=146), dict(lda=1 << 22), dict(ldb=1 << 22),
            dict(m=3, a=N), dict(m=3, sa=N), dict(m=3, b=N), dict(m=3, sb=N), dict(m=3, c=N),
            dict(m=3, a=_p(0x10008)), dict(m=3, b=_p(0x10008)), dict(m=3, c=_p(0x10004)),
            dict(m=3, sa=_p(0x10001)), dict(m=3, sb=_p(0x10002))]
GEMM = dict(a=_p(), lda=512, sa=_p(), b=_p(), ldb=512, sb=_p(), u=_p(), su=_p(), c=_p(), ldc=144,
            m=0, n=144, k=512, limit=7.0)


def test_dense_int8(lib):
    def call(**kw):
        a = {**GEMM, **kw}
        return lib.moe_dense_gemm_int8(a["a"], a["lda"], a["sa"], a["b"], a["ldb"], a["sb"], a["c"],
                                       a["ldc"], a["m"], a["n"], a["k"], N)
    assert call() == 0
    for kw in GEMM_BAD:
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"dense_gemm_int8"), kw


def test_swiglu_int8(lib):
    def call(**kw):
        a = {**GEMM, **kw}
        return lib.moe_dense_gate_up_swiglu_int8(
            a["a"], a["lda"], a["sa"], a["b"], a["sb"], a["u"], a["su"], a["ldb"], a["c"], a["ldc"],
            a["m"], a["n"], a["k"], a["limit"], N)
    assert call() == 0
    for kw in GEMM_BAD + [dict(limit=0.0), dict(limit=-1.0), dict(limit=NAN), dict(m=3, u=N),
                          dict(m=3, su=N), dict(m=3, u=_p(0x10008)), dict(m=3, su=_p(0x10002))]:
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"dense_gate_up_swiglu_int8"), kw


def test_shared_expert_int8(lib):
    base = dict(a=_p(), lda=512, sa=_p(), g=_p(), sg=_p(), u=_p(), su=_p(), ldw=512, d=_p(),
                ldd=144, sd=_p(), o=_p(), ldo=512, m=0, inter=144, hidden=512, limit=7.0, ws=_p(),
                wb=1 << 40)

    def call(**kw):
        a = {**base, **kw}
        return lib.moe_shared_expert_int8(
            a["a"], a["lda"], a["sa"], a["g"], a["sg"], a["u"], a["su"], a["ldw"], a["d"], a["ldd"],
            a["sd"], a["o"], a["ldo"], a["m"], a["inter"], a["hidden"], a["limit"], a["ws"],
            a["wb"], N)
    assert call() == 0
    need = lib.moe_shared_expert_int8_workspace_bytes(3, 144)
    assert need >= 3 * 144 * 5 + 12
    for kw in (dict(m=-1), dict(m=1 << 22), dict(inter=136), dict(inter=0), dict(hidden=520),
               dict(lda=496), dict(ldw=500), dict(ldd=128), dict(ldo=256), dict(limit=0.0),
               dict(m=3, a=N), dict(m=3, sa=N), dict(m=3, g=N), dict(m=3, sg=N), dict(m=3, u=N),
               dict(m=3, su=N), dict(m=3, d=N), dict(m=3, sd=N), dict(m=3, o=N), dict(m=3, ws=N),
               dict(m=3, ws=_p(0x10010)), dict(m=3, d=_p(0x10008))):
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"shared_expert_int8"), kw
    assert call(m=3, wb=need - 1) == 2
    assert lib.moe_shared_expert_int8_workspace_bytes(0, 16) == 0
    assert lib.moe_shared_expert_int8_workspace_bytes(4, -16) == 0


def test_layer_few(lib):
    base = dict(x=_p(), ld_x=512, lg=N, ld_lg=0, bias=N, scale=1.0, renorm=1, ids=_p(), w=_p(),
                gp=_p(), gs=_p(), g2=_p(), dp=_p(), ds=_p(), d2=_p(), e=8, sh=N, ld_sh=0, o=_p(),
                ld_o=512, rows=0, top_k=2, hidden=512, mi=192, limit=7.0, ws=_p(), wb=1 << 40)

    def call(**kw):
        a = {**base, **kw}
        return lib.moe_w4a16_layer_few(*[a[n] for n in base], N)
    assert call() == 0
    assert call(lg=_p(), ld_lg=8, ids=N, w=N) == 0
    need = lib.moe_few_workspace_bytes(2, 2, 192)
    for kw in (dict(rows=-1), dict(rows=17), dict(top_k=0), dict(rows=16, top_k=17), dict(e=0),
               dict(hidden=0), dict(hidden=480, ld_x=512), dict(hidden=8256, ld_x=8256, ld_o=8256),
               dict(mi=0), dict(mi=160), dict(mi=65600), dict(limit=0.0), dict(limit=NAN),
               dict(ld_x=448), dict(ld_x=516), dict(ld_x=1 << 24), dict(ld_o=448), dict(ld_o=514),
               dict(sh=_p(), ld_sh=448), dict(sh=_p(), ld_sh=513), dict(lg=_p(), ld_lg=7),
               dict(lg=_p(), ld_lg=4096, e=2049), dict(lg=_p(), ld_lg=8, top_k=65),
               dict(lg=_p(), ld_lg=8, scale=INF), dict(lg=_p(), ld_lg=8, scale=NAN),
               dict(rows=2, x=N), dict(rows=2, o=N), dict(rows=2, ids=N), dict(rows=2, w=N),
               dict(rows=2, gp=N), dict(rows=2, gs=N), dict(rows=2, g2=N), dict(rows=2, dp=N),
               dict(rows=2, ds=N), dict(rows=2, d2=N), dict(rows=2, ws=N),
               dict(rows=2, x=_p(0x10008)), dict(rows=2, ws=_p(0x10008)), dict(rows=2, o=_p(0x10004)),
               dict(rows=2, sh=_p(0x10004), ld_sh=512)):
        assert call(**kw) == 1, kw
        assert lib.moe_w4a16_last_error().startswith(b"layer_few"), kw
    assert call(rows=2, wb=need - 1) == 2
    for args in ((0, 2, 64), (17, 1, 64), (16, 17, 64), (2, 0, 64), (2, 2, 0)):
        assert lib.moe_few_workspace_bytes(*args) == 0, args
    assert need >= 4 * 192 * 2 + 4 * 24 + 32

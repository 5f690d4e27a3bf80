"""More of what the feed-forward half's calls refuse on the host, and what their size queries say."""

import ctypes

import pytest

from test_ffn_library import N, lib  # noqa: F401


@pytest.mark.parametrize("rows,top_k,mi", [(2, 2, 100), (2, 2, 160), (1, 1, 32), (1, 8, 65600),
                                           (16, 16, 1 << 30), (1, 1, 2 ** 31 - 1)])
def test_a_few_workspace_of_widths_the_layer_does_not_take(lib, rows, top_k, mi):  # noqa: F811
    assert lib.moe_few_workspace_bytes(rows, top_k, mi) == 0


@pytest.mark.parametrize("mi", [64, 192, 65536])
def test_a_few_workspace_of_widths_the_layer_takes(lib, mi):  # noqa: F811
    assert lib.moe_few_workspace_bytes(16, 16, mi) >= 256 * (2 * mi + mi // 8 + 8)


def _norm(lib, form, **kw):
    """A call of 4 x 256 with made-up pointers; it must be refused (one that is launched reports so)."""
    a = dict(x=0x100000, ld_x=256, r=0x200000, ld_r=256, h=0x300000, ld_h=256, y=0x400000, ld_y=256)
    a.update(kw)
    p = ctypes.c_void_p
    args = [p(a["x"]), a["ld_x"], p(a["r"]), a["ld_r"], p(0x500000), 1e-6, p(a["h"]), a["ld_h"],
            p(a["y"]), a["ld_y"]]
    if form != "bf16":
        args += [p(0x600000), 256, p(0x700000)]
    if form == "fp8":
        args.append(2)
    return getattr(lib, "moe_rmsnorm_" + form)(*args, 4, 256, N), lib.moe_w4a16_last_error()


@pytest.mark.parametrize("form", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("kw,word", [
    (dict(h=0x100000, y=0x100000), b"h and y"), (dict(h=0x300000, y=0x300000), b"h and y"),
    (dict(h=0x100000, ld_h=264), b"leading"), (dict(h=0x200000, ld_r=264), b"leading"),
    (dict(y=0x100000, ld_x=512), b"leading")])
def test_a_norms_outputs_over_each_other_or_over_inputs_of_another_stride(lib, form, kw, word):  # noqa: F811
    """h and y are both stored: in one buffer (both may be x, each alone) one of them is lost. In
    place of an input with another leading dimension, a row's output lies over another row's input."""
    status, message = _norm(lib, form, **kw)
    assert status == 1 and word in message and message.startswith(b"rmsnorm_" + form.encode())

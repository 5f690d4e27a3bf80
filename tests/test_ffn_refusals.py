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

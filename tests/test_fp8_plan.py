"""The tile rule of the FP8 products: the measurements in its comment mark the tiles it takes, and
the GPU tests' lists reach every tile and split."""

import re

import fp8_plan
import test_gpu_fp8
import test_gpu_fp8_swiglu
from test_fp8_library import lib  # noqa: F401 (a fixture)


def _marked():
    """(swiglu, rows, experts, {column: marked}) of the comment's table; columns are (rows, weight
    rows) of a tile, or for the splits of K their number."""
    text = open(fp8_plan.SOURCE).read()
    table = text[text.index("//   plain,"):text.index("template <bool kSwiglu>\nFp8Plan")]
    head = None
    for line in table.splitlines():
        label, *cells = [c for c in re.split(r"\s{2,}", line.strip("/ ").strip()) if c]
        if label.startswith("("):
            break
        if "experts" not in label and "row" not in label:
            head = label, cells
            continue
        kind, cols = head[0].split(",")[0], head[1]
        assert len(cells) == len(cols), line
        experts = int(m.group(1)) if (m := re.match(r"(\d+) experts", label)) else 0
        rows = int(re.search(r"(\d+) rows?", label).group(1)) * max(experts, 1)
        tiles = [tuple(int(v) for v in reversed(c.split(" x "))) if " x " in c else int(c)
                 for c in cols]
        yield kind != "plain", rows, experts, {c: v.endswith("*") for c, v in zip(tiles, cells)}
    split = table[table.index("split of K"):].splitlines()
    ways = [int(v) for v in re.split(r"\s{2,}", split[0].strip())[1:]]
    for line in split[1:]:
        m = re.match(r"//\s+(\d+) rows, (\d+) x (\d+)\s+(.*)", line)
        if m:
            yield (int(m.group(3)), int(m.group(2))), int(m.group(1)), 0, \
                {w: v.endswith("*") for w, v in zip(ways, m.group(4).split())}


def test_the_comments_marks_are_the_tiles_taken():
    seen = 0
    for kind, rows, experts, cells in _marked():
        swiglu = kind is not False
        n, k = (2048, 6144) if swiglu else (6144, 2048)
        t, ways = fp8_plan.plan(swiglu, rows, experts, n, k, split=isinstance(kind, tuple))
        shape = fp8_plan.tile(swiglu, t)
        taken = ways if isinstance(kind, tuple) else shape
        assert [c for c, mark in cells.items() if mark] == [taken], (kind, rows, experts)
        if isinstance(kind, tuple):
            assert shape == kind
        seen += 1
    assert seen == 14


def test_the_library_splits_as_the_plan_says(lib):  # noqa: F811
    for rows in (1, 7, 64, 77, 256, 300, 1000, 4096):
        for experts in (0, 1, 8, 64, 256):
            for n, k in ((144, 2064), (1360, 1040), (2048, 6144), (768, 2048), (16, 16)):
                _, ways = fp8_plan.plan(True, rows, experts, n, k)
                want = ways * rows * n * 8 if ways > 1 else 0
                assert lib.moe_fp8_swiglu_workspace_bytes(rows, experts, n, k) == want


def test_the_plain_lists_reach_every_tile():
    dense = {fp8_plan.plan(False, m, 0, n, k)[0] for m, n, k in test_gpu_fp8.DENSE}
    grouped = {fp8_plan.plan(False, r, e, n, k)[0] for e, r, n, k, _ in test_gpu_fp8.GROUPED}
    assert dense == grouped == {0, 1, 2, 3}


def test_the_swiglu_lists_reach_every_tile_in_one_launch():
    dense = [fp8_plan.plan(True, m, 0, n, k) for m, n, k in test_gpu_fp8_swiglu.DENSE]
    grouped = [fp8_plan.plan(True, r, e, n, k) for e, r, n, k, _ in test_gpu_fp8_swiglu.GROUPED]
    for plans in (dense, grouped):
        assert {t for t, ways in plans if ways == 1} == {0, 1, 2, 3}


def test_the_split_lists_are_what_they_say():
    """Every tile in every number of splits it takes, dense and grouped (the dense 128-row tile
    is not split in two), and with an empty last split."""
    dense, grouped = test_gpu_fp8_swiglu.DENSE_SPLIT, test_gpu_fp8_swiglu.GROUPED_SPLIT
    for c in dense:
        assert fp8_plan.plan(True, c[2], 0, *c[3:]) == c[:2], c
    for c in grouped:
        assert fp8_plan.plan(True, c[3], c[2], *c[4:6]) == c[:2], c
    everything, empty = {(t, w) for t in range(4) for w in (2, 4, 8)}, set()
    assert {c[:2] for c in dense} == everything - {(2, 2)}
    assert {c[:2] for c in grouped} == everything
    for c in dense + grouped:
        blocks = -(-c[-1 if c in dense else 5] // 128)
        if -(-blocks // c[1]) * (c[1] - 1) >= blocks:
            empty.add((c[0], c in dense))
    assert empty == {(t, kind) for t in range(4) for kind in (True, False)} - {(2, False)}

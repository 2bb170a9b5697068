"""How attention deals its work to workgroups, on the kernels' own arithmetic
(compiled for the host): every tile of tokens of every item is taken once, and
the join finds what was left of it."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("split") / "split_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-fPIC", "-shared",
                    "-I" + os.path.join(ROOT, "entropy_coding_amd", "csrc"),
                    os.path.join(ROOT, "tests", "split_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def run(rows, contexts, heads, ratio, chain, tile_shift, unit_shift, unit_tokens, target, least):
        rows, contexts = np.asarray(rows, np.int32), np.asarray(contexts, np.int32)
        n_items = int((-(-rows.astype(np.int64) * ratio // (1 << tile_shift))).sum()) * heads
        parts = np.zeros((n_items + 2 * target + 1, 9), np.int32)
        items = np.zeros((n_items + 1, 6), np.int32)
        per, count = ctypes.c_uint32(0), ctypes.c_int(0)
        p = lambda x: x.ctypes.data_as(ctypes.c_void_p)
        n = lib.split_parts(len(rows), p(rows), p(contexts), heads, ratio, int(chain), tile_shift, unit_shift,
                            unit_tokens, target, least, ctypes.byref(per), p(parts), len(parts), p(items), len(items),
                            ctypes.byref(count))
        assert n >= 0 and count.value == n_items
        return per.value, parts[:n].tolist(), items[:n_items].tolist()

    run.slot = lambda first, last, s: lib.sharer_slot(first, last, s)
    run.full = lib.tile_full
    return run


def check(split, rows, contexts, heads, ratio, chain, tile_shift, unit_shift, unit_tokens, target, least):
    per, parts, items = split(rows, contexts, heads, ratio, chain, tile_shift, unit_shift, unit_tokens, target, least)
    by_item, slots = {}, {}
    for w, b, h, tile, ta, tb, whole, slot, length in parts:
        assert 0 <= w < target and ta <= tb
        by_item.setdefault((b, h, tile), []).append((w, ta, tb, whole, slot))
        if not whole:
            assert 0 <= slot < 2 * target and slot not in slots
            slots[slot] = (b, h, tile)
    assert len(by_item) == len(items)
    for b, h, tile, first, last, length in items:
        got = by_item[(b, h, tile)]
        # what a row tile sees, from the definition
        top = min((tile + 1) << tile_shift, int(rows[b]) * ratio) - 1
        assert length == int(contexts[b]) + (top // ratio + 1 if chain else int(rows[b]))
        assert got[0][1] == 0 and got[-1][2] == -(-length // unit_tokens)
        assert all(x[2] == y[1] and x[0] + 1 == y[0] for x, y in zip(got, got[1:]))
        if first == last:
            assert len(got) == 1 and got[0][3]
        else:
            assert last < target and not any(g[3] for g in got)
            assert [g[0] for g in got] == list(range(first, last + 1))
            assert [g[4] for g in got] == [split.slot(first, last, s) for s in range(last - first + 1)]
    return per, parts


@pytest.mark.parametrize("seed", range(120))
def test_every_tile_is_taken_once(split, seed):
    rng = np.random.default_rng(seed)
    batch, heads, ratio = int(rng.integers(1, 60)), int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 4, 5, 16]))
    wide = bool(rng.integers(2))
    tile_shift, unit_shift, least = (int(rng.choice([6, 7])), 6, 1) if wide else (4, 5, 4)
    rows = rng.integers(0, 300 if wide else 8, batch)
    contexts = rng.integers(0, int(rng.choice([50, 3000, 40000])) + 1, batch)
    check(split, rows, contexts, heads, ratio, bool(rng.integers(2)), tile_shift,
          unit_shift + int(rng.choice([0, 0, 1, 3])), 64 if wide else 32, int(rng.choice([256, 512, 768])), least)


@pytest.mark.parametrize("chain", [True, False])
@pytest.mark.parametrize("case", [
    # rows, contexts, heads, ratio, tile_shift, unit_shift, unit_tokens, target, least
    ([1], [0], 1, 1, 4, 5, 32, 1024, 4),
    ([1], [32767], 8, 4, 4, 5, 32, 512, 4),
    ([64], [32768], 8, 8, 7, 6, 64, 512, 1),
    ([1000, 1000], [7001, 7001], 8, 4, 7, 6, 64, 512, 1),
    ([1] * 2000, [0] * 2000, 8, 4, 4, 5, 32, 512, 4),
    ([0, 3, 0, 0, 5], [10, 0, 0, 9000, 1], 2, 2, 4, 5, 32, 768, 4),
    ([4096], [0], 2, 4, 7, 6, 64, 512, 1),
    ([70000], [3], 1, 1, 6, 6, 64, 256, 1),
    ([1], [(1 << 31) - 300], 1, 1, 4, 5, 32, 1024, 4),
    ([1, 900], [(1 << 31) - 300, 5], 1, 1, 7, 9, 64, 512, 1),
    ([2, 2], [(1 << 30), 1], 1, 1, 4, 31, 32, 512, 4),
])
def test_the_edges(split, case, chain):
    rows, contexts, heads, ratio, tile_shift, unit_shift, unit_tokens, target, least = case
    per, parts = check(split, rows, contexts, heads, ratio, chain, tile_shift, unit_shift, unit_tokens, target, least)
    # nobody has more than its share
    assert per >= least and max(p[0] for p in parts) < target


def test_rows_that_see_a_tile_in_full(split):
    """Tokens before `full` are seen by the first row of a tile, and so by
    all; the token there is not."""
    for chain in (1, 0):
        for context in (0, 5, 64):
            for ratio in (1, 3, 5, 16, 200):
                for nodes in (1, 7, 100):
                    for row0 in range(0, nodes * ratio, 64):
                        full = split.full(chain, context, nodes, row0, 64, ratio)
                        assert full == context + (row0 // ratio + 1 if chain else 0)

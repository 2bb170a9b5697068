"""The host-side checks of the paged cache's calls, with no GPU: bad
arguments are refused with the status their declarations state before
anything touches the device (device pointers are stand-in addresses that host
code must never dereference, so the module stays off machines with a GPU),
and a model of how the attention splits its work over workgroups."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_reference as R
from test_host_sanitizers import ROOT, _runtime, checked_lib  # noqa: F401  (a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="stand-in device pointers: host-only checks, kept off GPUs")

FAKE = 1 << 40


def paged_desc(kvc, **kw):
    f = dict(d_pools=FAKE, d_block_table=FAKE, n_pools=4, pool_bytes=10 * 16 * 8 * 128 * 2, batch=3, heads=8,
             max_pages=4, num_pages=10, page_tokens=16, reserved=0)
    f.update(kw)
    return kvc.kvc_paged_kv(**f)


def table_status(kvc, ws=FAKE, ws_bytes=None, **kw):
    f = dict(batch=3, max_pages=4, num_pages=10, free_capacity=10, max_rows=20, page_tokens=16, trim=0,
             d_cached_lens=FAKE, d_new_lens=FAKE, d_held_in=FAKE, d_held_out=FAKE, d_block_table=FAKE,
             d_free_pages=FAKE, d_free_in=FAKE, d_free_out=FAKE, d_row_starts=FAKE, d_slots=FAKE, d_positions=FAKE)
    f.update(kw)
    n = 256 + 12 * (f["batch"] + 64) if ws_bytes is None else ws_bytes
    return kvc._lib_block_table(ctypes.byref(kvc.kvc_block_table(**f)), ws, n, None, None)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(batch=1 << 31), dict(max_pages=0), dict(max_pages=1 << 31), dict(batch=1 << 16, max_pages=1 << 15),
    dict(num_pages=0), dict(num_pages=1 << 31), dict(free_capacity=-1), dict(free_capacity=1 << 31), dict(max_rows=-1),
    dict(max_rows=1 << 31), dict(page_tokens=0), dict(trim=2), dict(d_held_in=None), dict(d_held_out=None),
    dict(d_block_table=None), dict(d_free_pages=None), dict(d_free_in=None), dict(d_free_out=None),
    dict(d_row_starts=None), dict(d_cached_lens=FAKE + 2), dict(d_new_lens=FAKE + 1), dict(d_slots=FAKE + 4),
    dict(d_positions=FAKE + 2), dict(ws=None), dict(ws=FAKE + 128),
])
def test_block_table_refuses(kvc, bad):
    assert table_status(kvc, **bad) == kvc.KVC_ERR_INVALID


def test_block_table_refuses_a_short_workspace(kvc):
    assert table_status(kvc, ws_bytes=256 + 12 * 67 - 1) == kvc.KVC_ERR_CAPACITY
    assert kvc._lib_block_table(None, FAKE, 1 << 20, None, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_block_table_result(None, None, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_block_table_result(FAKE + 8, None, None) == kvc.KVC_ERR_INVALID


def append_status(kvc, layer=0, kv_dtype=0, ch=128, k=FAKE, v=FAKE, src=0, rows=5, ks=1024, vs=1024, slots=FAKE,
                  k_scale=1.0, v_scale=1.0, **kw):
    return kvc._lib_append(ctypes.byref(paged_desc(kvc, **kw)), layer, kv_dtype, ch, k, v, src, rows, ks, vs, slots,
                           k_scale, v_scale, None)


@pytest.mark.parametrize("bad", [
    dict(layer=-1), dict(layer=2), dict(n_pools=3), dict(n_pools=0), dict(kv_dtype=2), dict(src=2), dict(src=1),
    dict(ch=0), dict(ch=96), dict(heads=0), dict(num_pages=0), dict(num_pages=11), dict(page_tokens=0),
    dict(page_tokens=17), dict(d_pools=None), dict(d_pools=FAKE + 4), dict(reserved=1), dict(k=None), dict(v=None),
    dict(k=FAKE + 8), dict(v=FAKE + 2), dict(slots=None), dict(slots=FAKE + 4), dict(rows=-1), dict(rows=1 << 31),
    dict(ks=1023), dict(ks=1020), dict(vs=1016), dict(vs=-1024), dict(ks=1 << 41), dict(k_scale=0.5),
    dict(v_scale=math.nan), dict(kv_dtype=1, k_scale=0.0), dict(kv_dtype=1, v_scale=-1.0),
    dict(kv_dtype=1, k_scale=math.inf),
])
def test_append_refuses(kvc, bad):
    assert append_status(kvc, **bad) == kvc.KVC_ERR_INVALID


def test_append_of_no_rows_launches_nothing(kvc):
    assert append_status(kvc, rows=0, k=None, v=None, slots=None) == kvc.KVC_OK


def attention(kvc, **kw):
    f = dict(d_q=FAKE, q_row_stride=32 * 128, q_head_stride=128, d_out=FAKE, out_row_stride=32 * 128, d_lse=FAKE,
             d_row_starts=FAKE, d_context_lens=FAKE, d_tree_mask=FAKE, mask_words=1, rows=12, rows_per_sequence=4,
             max_tokens=64, q_heads=32, channels=128, kv_dtype=0, softmax_scale=0.1, k_scale=1.0, v_scale=1.0)
    f.update({k: v for k, v in kw.items() if k in f})
    return kvc.kvc_attention(**f), paged_desc(kvc, **{k: v for k, v in kw.items() if k not in f})


def attention_status(kvc, layer=0, ws=FAKE, ws_bytes=1 << 40, **kw):
    p, g = attention(kvc, **kw)
    return kvc._lib_attention(ctypes.byref(g), layer, ctypes.byref(p), ws, ws_bytes, None)


def sizes(kvc, **kw):
    p, g = attention(kvc, **kw)
    n = ctypes.c_uint64(0)
    return kvc._lib_attention_sizes(ctypes.byref(g), ctypes.byref(p), ctypes.byref(n)), n.value


SIZES_BAD = [
    dict(channels=32), dict(channels=320), dict(channels=96), dict(kv_dtype=2), dict(kv_dtype=-1), dict(rows=-1),
    dict(rows=1 << 24), dict(rows_per_sequence=-1), dict(max_tokens=-1), dict(q_heads=0), dict(q_heads=30),
    dict(q_heads=8 * 1025), dict(softmax_scale=math.nan), dict(softmax_scale=math.inf), dict(k_scale=0.0),
    dict(v_scale=-2.0), dict(batch=0), dict(batch=(1 << 20) + 1), dict(max_pages=0), dict(heads=0),
    dict(page_tokens=0), dict(num_pages=11), dict(num_pages=1 << 28, pool_bytes=1 << 62), dict(reserved=3),
    dict(n_pools=1), dict(d_pools=None), dict(batch=(1 << 14) + 1), dict(softmax_scale=3e38),
    dict(softmax_scale=1e30, k_scale=1e30),
]


@pytest.mark.parametrize("bad", SIZES_BAD + [
    dict(layer=-1), dict(layer=2), dict(d_q=None), dict(d_q=FAKE + 8), dict(d_out=None), dict(d_out=FAKE + 2),
    dict(q_row_stride=4), dict(q_row_stride=-8), dict(q_head_stride=12), dict(out_row_stride=32 * 128 - 8),
    dict(out_row_stride=32 * 128 + 4), dict(d_lse=FAKE + 2), dict(d_row_starts=None), dict(d_row_starts=FAKE + 2),
    dict(d_context_lens=FAKE + 2), dict(d_tree_mask=FAKE + 4), dict(mask_words=0), dict(mask_words=(1 << 20) + 1),
    dict(d_tree_mask=None, mask_words=1), dict(d_block_table=None), dict(d_block_table=FAKE + 2), dict(ws=None),
    dict(ws=FAKE + 128),
])
def test_attention_refuses(kvc, bad):
    assert attention_status(kvc, **bad) == kvc.KVC_ERR_INVALID


@pytest.mark.parametrize("bad", SIZES_BAD)
def test_attention_sizes_refuse(kvc, bad):
    assert sizes(kvc, **bad)[0] == kvc.KVC_ERR_INVALID


def test_attention_sizes_and_a_short_workspace(kvc):
    st, n = sizes(kvc)
    assert st == kvc.KVC_OK and n % 256 == 0
    assert attention_status(kvc, ws_bytes=n - 1) == kvc.KVC_ERR_CAPACITY
    # with a launch shape of its own, a call of fewer rows needs no more
    for ratio in (1, 4, 8):
        for hint in (1, 5, 64):
            last = 0
            for rows in (0, 1, 2, 3, 7, 12, 40, 300, 5000):
                st, n = sizes(kvc, rows=rows, rows_per_sequence=hint, q_heads=8 * ratio, max_tokens=0, max_pages=4000)
                assert st == kvc.KVC_OK and n >= last
                last = n
    assert kvc._lib_attention_result(None, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_attention_result(FAKE + 64, None) == kvc.KVC_ERR_INVALID


def split_model(lens, rows, heads, ratio, tile_rows, unit, target, least):
    """The attention's split in Python: the parts (sequence, head, row tile,
    first tile, last tile, whole, slot) of every workgroup."""
    tiles = [-(-r * ratio // tile_rows) for r in rows]
    real = [-(-n // unit) for n in lens]
    total = sum(t * heads * u for t, u in zip(tiles, real))
    per = max(-(-total // target), least)
    aligned, tried = False, per
    for _ in range(2):
        if sum(t * heads * -(-u // tried) for t, u in zip(tiles, real)) <= target:
            aligned, per = True, tried
            break
        tried += (tried + 7) // 8
    items, base = [], 0
    for b, (t, u) in enumerate(zip(tiles, real)):
        size = -(-u // per) * per if aligned else u
        for i in range(t * heads):
            items.append((base, size, u, b, i // t, i % t))
            base += size
    parts = []
    for w in range(target):
        lo, hi = w * per, (w + 1) * per
        for first, size, u, b, h, tile in items:
            if first < hi and first + size > lo and size:
                at, to = max(first, lo), min(first + size, hi)
                parts.append((w, b, h, tile, min(at - first, u), min(to - first, u),
                              first >= lo and first + size <= hi, 2 * w + (first >= lo), u))
    return per, aligned, items, parts


@pytest.mark.parametrize("seed", range(40))
def test_the_attention_split_covers_every_token_once(seed):
    """Every tile of every item is in exactly one part; a workgroup leaves at
    most one part in each of its two places; the join finds an item's parts in
    the places it reads; no place lies outside the workspace."""
    rng = np.random.default_rng(seed)
    batch, heads, ratio = int(rng.integers(1, 60)), int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 4, 5]))
    wide = bool(rng.integers(2))
    tile_rows, unit, least = (128, 64, 1) if wide else (16, 32, 4)
    rows = rng.integers(0, 200 if wide else 5, batch)
    lens = rng.integers(0, int(rng.choice([50, 3000, 40000])), batch) + rows
    target = int(rng.choice([256, 512, 768]))
    per, aligned, items, parts = split_model(lens.tolist(), rows.tolist(), heads, ratio, tile_rows, unit, target, least)
    covered, places = {}, set()
    for w, b, h, tile, lo, hi, whole, slot, u in parts:
        covered.setdefault((b, h, tile), []).append((lo, hi, whole, slot))
        if not whole:
            assert slot not in places and slot < 2 * target
            places.add(slot)
    assert len(covered) == len([i for i in items if i[1]])
    for first, size, u, b, h, tile in items:
        if not size:
            continue
        got = sorted(covered[(b, h, tile)], key=lambda p: p[:2])
        assert got[0][0] == 0 and got[-1][1] == u and all(x[1] == y[0] for x, y in zip(got, got[1:]))
        w0, w1 = first // per, (first + size - 1) // per
        assert w1 < target
        if w0 == w1:
            assert len(got) == 1 and got[0][2]
        else:
            assert [p[3] for p in sorted(got, key=lambda p: p[3] // 2)] == [2 * w0 + 1] + [2 * w for w in range(w0 + 1, w1 + 1)]


def test_the_plain_block_table_conserves_pages():
    """The tests' reference itself: no page is lost or held twice, and
    trimming what a step took restores the stack."""
    rng = np.random.default_rng(3)
    for _ in range(50):
        batch, page = rng.integers(1, 9), int(rng.integers(1, 20))
        cached, new = rng.integers(0, 60, batch), rng.integers(0, 30, batch)
        held = -(-cached // page) + rng.integers(0, 3, batch)
        cap = int(max(held.max(), (-(-(cached + new) // page)).max()))
        pages = int(held.sum()) + 200
        perm = rng.permutation(pages).astype(np.int32)
        table = np.full((batch, cap), -1, np.int32)
        at = 0
        for b in range(batch):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        free = np.concatenate([perm[at:], np.full(at, -1, np.int32)])
        t, h, f, c, starts, slots, pos = R.block_table(table, held, free, pages - at, page, cached, new, 300, True)
        mine = np.concatenate([t[b, :h[b]] for b in range(batch)])
        assert sorted(np.concatenate([mine, f[:c]])) == list(range(pages))
        assert starts[-1] == new.sum() and len(set(slots[:starts[-1]])) == starts[-1] and (slots[starts[-1]:] == -1).all()
        t2, h2, f2, c2 = R.block_table(t, h, f, c, page, cached, np.zeros_like(new), 300, True)[:4]
        t3, h3, f3, c3 = R.block_table(t2, h2, f2, c2, page, cached, new, 300, True)[:4]
        assert c3 == c and np.array_equal(f3[:c], f[:c]) and np.array_equal(h3, h)


def test_paged_host_logic_under_the_sanitizers(checked_lib):  # noqa: F811
    """This module's refusals against the library whose host code is built
    with AddressSanitizer and UndefinedBehaviorSanitizer."""
    if os.environ.get("KVC_LIBRARY"):
        pytest.skip("already running on the sanitizer build")
    env = dict(os.environ)
    env["KVC_LIBRARY"] = checked_lib
    env["LD_PRELOAD"] = ":".join(p for p in [_runtime("libasan.so"), env.get("LD_PRELOAD", "")] if p)
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "tests/test_host_paged_ops.py", "-k", "not sanitizers"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "passed" in r.stdout, (r.stdout + r.stderr)[-4000:]
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-4000:]

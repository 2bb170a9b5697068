"""The host-side checks of the speculative step's calls, with no GPU: bad
arguments are refused with the status their declarations state before
anything touches the device (device pointers are stand-in addresses, so the
module stays off machines with a GPU)."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

from test_host_paged_ops import FAKE, paged_desc
from test_host_sanitizers import ROOT, _runtime, checked_lib  # noqa: F401  (a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="stand-in device pointers: host-only checks, kept off GPUs")


def qkv_status(kvc, layer=0, **kw):
    f = dict(d_q=FAKE, q_row_stride=48 * 128, q_head_stride=128, d_k=FAKE, k_row_stride=48 * 128, k_head_stride=128, d_v=FAKE,
             v_row_stride=48 * 128, v_head_stride=128, d_q_out=FAKE, q_out_row_stride=32 * 128, d_q_norm=FAKE, d_k_norm=FAKE,
             d_frequencies=FAKE, d_positions=FAKE, d_slots=FAKE, rows=5, q_heads=32, channels=128, rotary=128, kv_dtype=0,
             norm_dtype=0, neighbours=0, eps=1e-6, k_scale=1.0, v_scale=1.0)
    f.update({k: v for k, v in kw.items() if k in f})
    g = paged_desc(kvc, **{k: v for k, v in kw.items() if k not in f})
    return kvc._lib_qkv(ctypes.byref(g), layer, ctypes.byref(kvc.kvc_qkv(**f)), None)


@pytest.mark.parametrize("bad", [
    dict(layer=-1), dict(layer=2), dict(n_pools=3), dict(d_pools=None), dict(num_pages=11), dict(channels=96),
    dict(channels=320, pool_bytes=1 << 40), dict(channels=0), dict(kv_dtype=2), dict(rows=-1), dict(rows=1 << 31),
    dict(q_heads=-1), dict(q_heads=65537), dict(neighbours=2), dict(rotary=-16), dict(rotary=144), dict(rotary=8),
    dict(k_scale=0.0), dict(v_scale=math.nan), dict(k_scale=0.5), dict(kv_dtype=1, v_scale=-1.0), dict(norm_dtype=1),
    dict(norm_dtype=3), dict(d_q_norm=FAKE + 8), dict(d_k_norm=FAKE + 2), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf),
    dict(eps=-1e-6), dict(eps=1e-31), dict(d_q_norm=None, eps=0.0), dict(d_frequencies=None), dict(d_frequencies=FAKE + 4),
    dict(d_positions=None), dict(d_positions=FAKE + 2), dict(d_q=None), dict(d_q=FAKE + 8), dict(d_k=None), dict(d_k=FAKE + 2),
    dict(d_v=None), dict(d_v=FAKE + 8), dict(d_slots=None), dict(d_slots=FAKE + 4), dict(d_q_out=None), dict(d_q_out=FAKE + 8),
    dict(q_row_stride=4), dict(q_row_stride=-8), dict(q_head_stride=12), dict(k_row_stride=-8), dict(k_head_stride=4),
    dict(v_row_stride=1 << 41), dict(v_head_stride=2), dict(q_out_row_stride=32 * 128 - 8), dict(q_out_row_stride=32 * 128 + 4),
    dict(reserved=1),
])
def test_qkv_refuses(kvc, bad):
    assert qkv_status(kvc, **bad) == kvc.KVC_ERR_INVALID


def test_qkv_of_no_rows_launches_nothing(kvc):
    assert qkv_status(kvc, rows=0, d_q=None, d_k=None, d_v=None, d_slots=None, d_q_out=None) == kvc.KVC_OK
    assert kvc._lib_qkv(ctypes.byref(paged_desc(kvc)), 0, None, None) == kvc.KVC_ERR_INVALID


def verify_status(kvc, ws=FAKE, ws_bytes=1 << 40, sizes=False, **kw):
    f = dict(batch=3, rows=12, vocab=1000, d_row_starts=FAKE, d_tokens=FAKE, d_parents=FAKE, d_target=FAKE,
             target_row_stride=1000, d_draft=FAKE, draft_row_stride=1003, d_accept=FAKE, d_sample=FAKE, d_kept=FAKE,
             d_kept_lens=FAKE, d_out_tokens=FAKE)
    f.update(kw)
    p = ctypes.byref(kvc.kvc_drafts(**f))
    if sizes:
        n = ctypes.c_uint64(0)
        return kvc._lib_verify_sizes(p, ctypes.byref(n)), n.value
    return kvc._lib_verify(p, ws, ws_bytes, None)


VERIFY_SIZES_BAD = [dict(batch=0), dict(batch=(1 << 20) + 1), dict(rows=-1), dict(rows=1 << 31), dict(vocab=0),
                    dict(vocab=(1 << 20) + 1), dict(batch=1 << 16, vocab=1 << 20), dict(batch=1 << 20, vocab=65536)]


@pytest.mark.parametrize("bad", VERIFY_SIZES_BAD + [
    dict(d_row_starts=None), dict(d_tokens=None), dict(d_target=None), dict(d_accept=None), dict(d_sample=None),
    dict(d_kept=None), dict(d_kept_lens=None), dict(d_out_tokens=None), dict(d_row_starts=FAKE + 2), dict(d_tokens=FAKE + 1),
    dict(d_parents=FAKE + 2), dict(d_target=FAKE + 2), dict(d_draft=FAKE + 1), dict(d_accept=FAKE + 2), dict(d_sample=FAKE + 3),
    dict(d_kept=FAKE + 2), dict(d_kept_lens=FAKE + 2), dict(d_out_tokens=FAKE + 2), dict(target_row_stride=999),
    dict(target_row_stride=1 << 41), dict(draft_row_stride=0), dict(draft_row_stride=-1000), dict(ws=None), dict(ws=FAKE + 128),
])
def test_verify_refuses(kvc, bad):
    assert verify_status(kvc, **bad) == kvc.KVC_ERR_INVALID


def test_verify_sizes_and_a_short_workspace(kvc):
    for bad in VERIFY_SIZES_BAD:
        assert verify_status(kvc, sizes=True, **bad)[0] == kvc.KVC_ERR_INVALID
    last = 0
    for kw in (dict(rows=0), dict(rows=10 ** 6, vocab=1 << 20),
               dict(batch=(1 << 16) - 1, rows=(1 << 31) - 1, vocab=1 << 20)):
        kw.update(target_row_stride=1 << 20, draft_row_stride=1 << 20)
        st, n = verify_status(kvc, sizes=True, **kw)
        assert st == kvc.KVC_OK and n > last
        last = n
        assert verify_status(kvc, ws_bytes=n - 1, **kw) == kvc.KVC_ERR_CAPACITY
    assert kvc._lib_verify(None, FAKE, 1 << 30, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_verify_result(None, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_verify_result(FAKE + 8, None) == kvc.KVC_ERR_INVALID


def compact_status(kvc, ws=FAKE, ws_bytes=256 + 12, kv_dtype=0, ch=128, rows=12, starts=FAKE, context=FAKE, kept=FAKE,
                   lens=FAKE, **kw):
    return kvc._lib_compact(ctypes.byref(paged_desc(kvc, **kw)), kv_dtype, ch, rows, starts, context, kept, lens, ws, ws_bytes,
                            None)


PAGES_BAD = [dict(n_pools=3), dict(n_pools=0), dict(n_pools=(1 << 20) + 2), dict(kv_dtype=2), dict(ch=0), dict(ch=96),
             dict(heads=0), dict(num_pages=0), dict(num_pages=11), dict(page_tokens=0), dict(d_pools=None), dict(d_pools=FAKE + 4),
             dict(reserved=1), dict(batch=0), dict(max_pages=0), dict(max_pages=1 << 31), dict(ws=None), dict(ws=FAKE + 64)]


@pytest.mark.parametrize("bad", PAGES_BAD + [
    dict(batch=(1 << 20) + 1), dict(rows=-1), dict(rows=1 << 31), dict(starts=None), dict(kept=None), dict(lens=None),
    dict(starts=FAKE + 2), dict(context=FAKE + 2), dict(kept=FAKE + 1), dict(lens=FAKE + 2), dict(d_block_table=None),
    dict(d_block_table=FAKE + 2),
])
def test_compact_refuses(kvc, bad):
    assert compact_status(kvc, **bad) == kvc.KVC_ERR_INVALID


def test_compact_refuses_a_short_workspace(kvc):
    assert compact_status(kvc, ws_bytes=256 + 11) == kvc.KVC_ERR_CAPACITY
    assert kvc._lib_compact_result(None, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_compact_result(FAKE + 8, None) == kvc.KVC_ERR_INVALID


def shared_status(kvc, fork, ws=FAKE, ws_bytes=256 + 4096 + 64, kv_dtype=0, ch=128, count=3, parents=FAKE, children=FAKE,
                  context=FAKE, **kw):
    f = dict(free_capacity=10, d_table=FAKE, d_held_in=FAKE, d_held_out=FAKE, d_free_pages=FAKE, d_free_in=FAKE,
             d_free_out=FAKE, d_extra=FAKE)
    f.update({k: v for k, v in kw.items() if k in f})
    f["d_block_table"] = f.pop("d_table")
    g = ctypes.byref(paged_desc(kvc, **{k: v for k, v in kw.items() if k not in f and k != "d_table"}))
    p = ctypes.byref(kvc.kvc_shared_pages(**f))
    if fork:
        return kvc._lib_fork(g, kv_dtype, ch, p, count, parents, children, context, ws, ws_bytes, None)
    return kvc._lib_release(g, kv_dtype, ch, p, count, children, ws, ws_bytes, None)


@pytest.mark.parametrize("fork", [True, False])
@pytest.mark.parametrize("bad", PAGES_BAD + [
    dict(count=-1), dict(count=1025), dict(children=None), dict(children=FAKE + 2), dict(free_capacity=9),
    dict(free_capacity=1 << 31), dict(d_table=None), dict(d_held_in=None), dict(d_held_out=None), dict(d_free_pages=None),
    dict(d_free_in=None), dict(d_free_out=None), dict(d_extra=None), dict(d_table=FAKE + 2), dict(d_held_in=FAKE + 1),
    dict(d_held_out=FAKE + 2), dict(d_free_pages=FAKE + 2), dict(d_free_in=FAKE + 2), dict(d_free_out=FAKE + 2),
    dict(d_extra=FAKE + 3),
])
def test_shared_pages_refuse(kvc, fork, bad):
    assert shared_status(kvc, fork, **bad) == kvc.KVC_ERR_INVALID


def test_forks_refuse(kvc):
    for bad in (dict(parents=None), dict(parents=FAKE + 2), dict(context=FAKE + 2)):
        assert shared_status(kvc, True, **bad) == kvc.KVC_ERR_INVALID
    for fork in (True, False):
        assert shared_status(kvc, fork, ws_bytes=256 + 4096 + 63) == kvc.KVC_ERR_CAPACITY
    assert kvc._lib_shared_result(None, None) == kvc.KVC_ERR_INVALID
    assert kvc._lib_shared_result(FAKE + 128, None) == kvc.KVC_ERR_INVALID


def test_step_host_logic_under_the_sanitizers(checked_lib):  # noqa: F811
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
                        "tests/test_host_step_ops.py", "-k", "not sanitizers"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "passed" in r.stdout, (r.stdout + r.stderr)[-4000:]
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-4000:]

"""The largest shapes that the paged cache's attention takes and the first
that it refuses, with no GPU (device pointers are stand-in addresses)."""
import pytest
import torch

from test_host_paged_ops import attention_status, sizes

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="stand-in device pointers: host-only checks, kept off GPUs")


def shape(heads, batch, rows, ratio=1, **kw):
    f = dict(heads=heads, q_heads=heads * ratio, batch=batch, rows=rows, channels=64, num_pages=1, page_tokens=16,
             pool_bytes=heads * 64 * 2 * 16, max_tokens=0, rows_per_sequence=0, q_row_stride=heads * ratio * 64,
             q_head_stride=64, out_row_stride=heads * ratio * 64)
    f.update(kw)
    return f


def items(heads, batch, rows, ratio=1):
    return heads * (rows * ratio // 16 + min(rows, batch))


@pytest.mark.parametrize("args", [(65536, 16384, 16384), (65536, 16384, 16383), (62000, 16384, 30000)])
def test_too_many_items_are_refused(kvc, args):
    assert items(*args) >= 1 << 30
    for kw in (dict(), dict(rows_per_sequence=64), dict(max_pages=1 << 30)):
        assert sizes(kvc, **shape(*args, **kw))[0] == kvc.KVC_ERR_INVALID
        assert attention_status(kvc, **shape(*args, **kw)) == kvc.KVC_ERR_INVALID


@pytest.mark.parametrize("args", [(61440, 16384, 16384), (65536, 1024, 32767), (1, 1, (1 << 24) - 1),
                                  (8, 16384, 16384, 1024 // 64)])
@pytest.mark.parametrize("max_pages", [1, 1 << 20, (1 << 31) - 1])
def test_the_largest_shapes_have_a_size(kvc, args, max_pages):
    """... at every width of the table, and one that the chip's workgroups
    bound where a sequence is long."""
    assert items(*args) < 1 << 30
    for hint in (0, 1, 64):
        st, n = sizes(kvc, **shape(*args, max_pages=max_pages, rows_per_sequence=hint))
        assert st == kvc.KVC_OK
        if max_pages > 1:
            assert n < 1 << 28


def test_widths_past_31_bits_change_nothing(kvc):
    """A table wider than any sequence: as the widest that one can fill."""
    wide = [sizes(kvc, **shape(8, 100, 100, max_pages=m, page_tokens=p, pool_bytes=1 << 50))
            for m, p in (((1 << 31) - 1, 1), ((1 << 31) - 1, 1 << 20), ((1 << 31) - 1, 1 << 21))]
    assert wide[0][0] == kvc.KVC_OK and len(set(wide)) == 1


def test_items_past_a_launch_are_dealt(kvc):
    """2^24 items of short sequences are more than a launch has workgroups
    for: the workspace is that of a dealt call."""
    st, n = sizes(kvc, **shape(16384, 1024, 1024, max_pages=4))
    assert st == kvc.KVC_OK and n < 1 << 26
    st, n = sizes(kvc, **shape(15000, 1000, 1000, max_pages=4))
    assert st == kvc.KVC_OK and n > 4 * 15000 * 1000


@pytest.mark.parametrize("hint", [1 << 24, 1 << 40, (1 << 61) + 1, (1 << 63) - 1])
def test_any_usual_number_of_rows(kvc, hint):
    """A hint of more rows than there can be is one of many rows."""
    for ratio in (1, 4, 1000):
        f = shape(2, 3, 4000 if ratio < 1000 else 20, ratio, max_pages=1000)
        assert sizes(kvc, **dict(f, rows_per_sequence=hint)) == sizes(kvc, **dict(f, rows_per_sequence=1 << 20))

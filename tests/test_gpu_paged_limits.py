"""Calls at the edge of what the paged cache's operators take."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_items_than_a_launch_has_workgroups_for(kvc, cuda):
    """1024 sequences of 16384 KV heads, one token each: a row sees that token
    alone, and its output is the token's V, bit for bit."""
    batch, heads, d = 1024, 16384, 64
    g = torch.Generator(device=cuda).manual_seed(61)
    v = torch.randn((batch, 1, heads, d), generator=g, device=cuda, dtype=torch.bfloat16)
    table = torch.randperm(batch, generator=g, device=cuda).to(torch.int32)[:, None]
    q = torch.randn((batch, heads, d), generator=g, device=cuda, dtype=torch.bfloat16)
    paged = kvc.PagedKV([q.view(batch, 1, heads, d), v], table, 1)
    starts = torch.arange(batch + 1, dtype=torch.int32, device=cuda)
    out, lse = kvc.kvc_paged_attention(paged, 0, q, starts)
    assert torch.equal(out, v[table[:, 0].long(), 0])
    k = paged.pools[0][table[:, 0].long(), 0].float()
    # 64 products of up to 6 x 6 summed in float32, scaled
    assert ((q.float() * k).sum(-1) * d ** -0.5 - lse).abs().max() < 80 * 2.0 ** -24 * 64 * 36 / 8


def test_a_stack_of_31_bits_with_surplus_pages(kvc, cuda):
    """2^31 - 1 free pages and two surplus ones that the step would take
    again: the state names more pages than there are, and stays as it is."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
    free = torch.empty((1 << 31) - 1, dtype=torch.int32, device=cuda)
    free[-4:] = i32([3, 4, 5, 6])
    count, held, table = i32([(1 << 31) - 1]), i32([3, 0]), i32([[7, 8, 9], [-1, -1, -1]])
    starts, slots = i32([0, 0, 0]), torch.zeros(40, dtype=torch.int64, device=cuda)
    tab = kvc.BlockTable(table, held, free, count, 16, (1 << 31) - 1, starts, slots)
    tab(i32([16, 0]), i32([0, 20]), trim=True)
    with pytest.raises(kvc.KvcError) as e:
        tab.result()
    assert e.value.status == kvc.KVC_ERR_INVALID
    assert int(count) == (1 << 31) - 1 and held.tolist() == [3, 0] and table.tolist() == [[7, 8, 9], [-1, -1, -1]]
    assert free[-4:].tolist() == [3, 4, 5, 6] and starts.tolist() == [0, 0, 0] and (slots == -1).all()
    # and one page fewer on the stack is a step like any other: its last page and the surplus ones
    count -= 2
    tab(i32([16, 0]), i32([0, 20]), trim=True)
    assert tab.result() == 20
    assert int(count) == (1 << 31) - 3 and held.tolist() == [1, 2] and table.tolist()[1][:2] == [8, 9]
    assert slots[:20].tolist() == [8 * 16 + i for i in range(16)] + [9 * 16 + i for i in range(4)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pools_that_are_not_16_byte_aligned_are_refused(kvc, cuda, kind):
    """Rows are written, and K is read, 16 bytes at a time."""
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    flat = [torch.zeros(4 * 16 * 2 * 64 + 8, dtype=dtype, device=cuda) for _ in range(2)]
    k = torch.zeros((1, 2, 64), dtype=dtype, device=cuda)
    slots, table = torch.zeros(1, dtype=torch.int64, device=cuda), torch.zeros((1, 4), dtype=torch.int32, device=cuda)
    for first, good in ((0, True), (1, False), (4, False)):
        pools = [flat[0][:4 * 16 * 2 * 64].view(4, 16, 2, 64), flat[1][first:first + 4 * 16 * 2 * 64].view(4, 16, 2, 64)]
        paged = kvc.PagedKV(pools, table, 16)
        if good:
            kvc.kvc_paged_append(paged, 0, k, k, slots)
            kvc.PagedAttention(paged, 2, 1)
            continue
        with pytest.raises(ValueError):
            kvc.kvc_paged_append(paged, 0, k, k, slots)
        with pytest.raises(ValueError):
            kvc.PagedAttention(paged, 2, 1)

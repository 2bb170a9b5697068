"""Objects of the paged cache that are made, called and dropped on different
streams, and made within a capture: their workspaces are theirs alone."""
import numpy as np
import pytest
import torch

import paged_reference as R
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000                             # tens of ms of a kernel that only counts cycles


class Step:
    """A block table's step of three requests with its expected outcome."""

    def __init__(self, cuda):
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
        self.cached, self.new = np.array([5, 0, 40]), np.array([7, 33, 1])
        table, held = np.full((3, 6), -1, np.int32), np.array([1, 0, 3], np.int32)
        table[0, 0], table[2, :3] = 9, [4, 2, 7]
        free = np.array([11, 8, 1, 0, 10, 3, 6, 5], np.int32)
        self.want = R.block_table(table, held, free, 8, 16, self.cached, self.new, 50, False)
        self.state = dev(table.tolist()), dev(held.tolist()), dev(free.tolist()), dev([8])
        self.starts = torch.zeros(4, dtype=torch.int32, device=cuda)
        self.slots = torch.zeros(50, dtype=torch.int64, device=cuda)
        self.lens = dev(self.cached.tolist()), dev(self.new.tolist())

    def table(self, kvc):
        return kvc.BlockTable(*self.state, 16, 12, self.starts, self.slots)

    def check(self):
        table, held, free, count, starts, slots = self.want[:6]
        assert np.array_equal(self.state[0].cpu(), table) and np.array_equal(self.state[1].cpu(), held)
        assert int(self.state[3]) == count and np.array_equal(self.state[2].cpu()[:count], free[:count])
        assert np.array_equal(self.starts.cpu(), starts) and np.array_equal(self.slots.cpu(), slots)


def attention_case(kvc, cuda):
    c = Case(kvc, cuda, [3000, 500], [9, 2], 2, 4, 128, "bf16", 16, True, seed=51)
    return c, (c.q, c.dev(c.starts), c.dev(c.contexts), c.dev(c.mask, torch.int64))


def test_made_behind_other_work_called_on_another_stream(kvc, cuda):
    step, side = Step(cuda), torch.cuda.Stream()
    c, args = attention_case(kvc, cuda)
    paged, ref = c.paged(), c.ref()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    tab, att = step.table(kvc), kvc.PagedAttention(paged, 8, len(c.q))
    torch.cuda._sleep(CYCLES)
    tab(*step.lens, stream=side)
    got = att(1, *args, stream=side)
    assert tab.result(side) == 41
    att.result(side)
    torch.cuda.synchronize()                     # whatever was still queued at construction
    step.check()
    c.check(got, ref)
    assert tab.result(side) == 41                # (the outcome, too, is still there)
    att.result(side)


@pytest.mark.parametrize("explicit", [True, False])
def test_dropped_while_a_call_is_queued(kvc, cuda, explicit):
    """The memory of an object that is dropped before its call has run goes to
    nobody else until it has."""
    step, side = Step(cuda), torch.cuda.Stream()
    c, args = attention_case(kvc, cuda)
    k = c.q[:, :2].contiguous()
    # pages that no sequence has
    unused = set(range(c.pools[0].shape[0])) - set(c.table[0, :189].tolist()) - set(c.table[1, :32].tolist())
    slots = torch.arange(len(k), device=cuda) + 16 * min(unused)
    ref = c.ref()
    torch.cuda.synchronize()
    tab, paged = step.table(kvc), c.paged()
    att = kvc.PagedAttention(paged, 8, len(c.q))
    kept = paged.block_table                     # the caller's own tensors outlive the work
    sizes = [tab.workspace.numel(), att.workspace.numel(), 8 * paged.ptrs.numel()]
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    kw = dict(stream=side) if explicit else {}
    with torch.cuda.stream(None if explicit else side):
        tab(*step.lens, **kw)
        kvc.kvc_paged_append(paged, 0, k, k, slots, **kw)
        got = att(1, *args, **kw)
    del tab, att, paged
    other = [torch.full((n,), 255, dtype=torch.uint8, device=cuda) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    step.check()
    assert np.array_equal(kept.cpu(), c.table)
    c.check(got, ref)
    assert torch.equal(c.pools[0].view(-1, 2, 128)[slots], k)
    assert all(bool((t == 255).all()) for t in other)


def test_made_within_a_capture(kvc, cuda):
    c, args = attention_case(kvc, cuda)
    paged, ref = c.paged(), c.ref()
    kvc.kvc_paged_attention(paged, 1, *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att = kvc.PagedAttention(paged, 8, len(c.q))
        got = att(1, *args)
    for _ in range(3):
        got[0].fill_(3.0)
        graph.replay()
        att.result()
        c.check(got, ref)
        torch.cuda.synchronize()

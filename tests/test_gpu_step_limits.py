"""The speculative step's calls at sizes where workgroups take several turns:
long rows of a table, wide pools, many pools; and their objects made, called
and dropped on different streams."""
import numpy as np
import pytest
import torch

import step_reference as S
from test_gpu_paged_share import Cache, dev
from test_gpu_verify_drafts import Case

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000                             # tens of ms of a kernel that only counts cycles


def test_a_very_long_prompt(kvc, cuda):
    """70000 pages of one token: forked, forked again, released."""
    lens = np.array([70000, 69999, 0, 0, 0, 0])
    c = Cache(kvc, cuda, [70000, 69999, 0, 0, 0, 0], 1, 1, 1, 64, "e4m3", 1, spare=40)
    c.share()
    c.fork([0, 1, 0, 1], [2, 3, 4, 5], lens)
    c.release([0, 2, 5])
    c.release([4, 1, 3])
    assert c.count == c.num_pages and not c.extra.any()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_forks_of_wide_pages(kvc, cuda, kind):
    """255 tokens of 130 pools to a child: 67 MB and more."""
    c = Cache(kvc, cuda, [2, 1, 0, 0, 0], 256, 65, 8, 128, kind, 2, spare=4)
    c.share()
    c.fork([0, 1, 0], [2, 3, 4], np.array([511, 255, 0, 0, 0]))
    c.release([2, 4])


def test_compaction_of_many_pools(kvc, cuda):
    """2100 pools: more columns than a sequence's workgroups have threads."""
    c = Cache(kvc, cuda, [1, 2], 16, 1050, 8, 128, "bf16", 3, spare=0)
    starts, context = np.array([0, 9, 25], np.int32), np.array([4, 3], np.int32)
    kept, lens = np.full(25, -1, np.int32), np.array([5, 12], np.int32)
    kept[:5], kept[9:21] = [0, 2, 3, 7, 8], [1, 2, 3, 4, 6, 7, 8, 9, 10, 11, 13, 15]
    op = kvc.PagedCompaction(c.paged)
    op(*(dev(x, cuda) for x in (starts, context, kept, lens)))
    op.result()
    S.compact(c.pools.numpy(), c.table, 16, starts, context, kept, lens)
    c.same_pools()


def test_large_batches(kvc, cuda):
    """Thousands of sequences: verification and compaction."""
    rng = np.random.default_rng(4)
    nodes = rng.integers(0, 4, 3000)
    Case(nodes, 50, True, 2, 5).run(kvc, cuda)
    Case(nodes, 50, False, 2, 6).run(kvc, cuda)
    Case(nodes[:1500], 5000, True, 0, 7).run(kvc, cuda)
    context = rng.integers(0, 3, 3000)
    c = Cache(kvc, cuda, (-(-(context + nodes) // 2)).tolist(), 2, 1, 1, 64, "e4m3", 8)
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    kept, lens = np.full(int(starts[-1]), -1, np.int32), rng.integers(0, nodes + 1).astype(np.int32)
    for b in range(3000):
        kept[starts[b]:starts[b] + lens[b]] = np.sort(rng.choice(nodes[b], lens[b], replace=False)) if lens[b] else []
    op = kvc.PagedCompaction(c.paged)
    op(dev(starts, cuda), dev(context.astype(np.int32), cuda), dev(kept, cuda), dev(lens, cuda))
    op.result()
    S.compact(c.pools.numpy(), c.table, 2, starts, context, kept, lens)
    c.same_pools()


class Work:
    """One call of every object, and what it has to give."""

    def __init__(self, kvc, cuda, seed):
        self.kvc, self.cuda = kvc, cuda
        self.case = Case([7, 3, 12], 9000, True, 3, seed)
        self.args = self.case.args(cuda)
        self.cache = Cache(kvc, cuda, [3, 2, 0, 0], 16, 2, 2, 64, "bf16", seed)
        self.cache.share()
        self.held, self.free, self.count, self.extra = self.cache.state
        self.lens = np.array([40, 25, 0, 0])
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
        self.fork_args = i32([0, 1]), i32([2, 3]), i32(self.lens.tolist())
        self.compact_args = i32([0, 9, 14, 14, 14]), i32([20, 8, 0, 0]), i32([0, 3, 4] + [-1] * 6 + [1, 2] + [-1] * 3), i32([3, 2, 0, 0])
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.q, self.k = (torch.randn((20, n, 64), generator=g).to(torch.bfloat16).to(cuda) for n in (4, 2))
        self.slots = torch.full((20,), -1, dtype=torch.int64, device=cuda)
        self.positions = torch.arange(20, dtype=torch.int32, device=cuda)
        self.freq = 100.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
        self.norm = torch.ones((2, 64))

    def make(self):
        c = self.cache
        return (self.kvc.DraftVerifier(3, 9000, 22), self.kvc.PagedCompaction(c.paged),
                self.kvc.SharedPages(c.paged, self.held, self.free, self.count, self.extra),
                self.kvc.PagedQKV(c.paged, 4, self.freq.to(self.cuda), self.norm.to(self.cuda), self.norm.to(self.cuda)))

    def call(self, made, **kw):
        verify, compact, shared, qkv = made
        self.got = verify(**self.args, **kw)
        compact(*self.compact_args, **kw)
        shared.fork(*self.fork_args, **kw)
        self.rotated = qkv(1, self.q, self.k, self.k, self.slots, self.positions, **kw)

    def check(self):
        self.case.check(self.got)
        c = self.cache
        S.compact(c.pools.numpy(), c.table, 16, np.array([0, 9, 14]), np.array([20, 8]), self.compact_args[2].cpu().numpy(), [3, 2])
        c.table, c.held, c.count, c.extra = S.fork(c.pools.numpy(), c.table, c.held, c.free, c.count, c.extra, 16, [0, 1], [2, 3],
                                                   self.lens)
        for got, want in ((c.t_table, c.table), (self.held, c.held), (self.count, [c.count]), (self.extra, c.extra)):
            assert np.array_equal(got.cpu().numpy(), want)
        c.same_pools()
        y, size = S.norm_rotate(S.f64(self.q), np.ones(64), 1e-6, np.arange(20), self.freq.numpy(), False)
        assert (np.abs(S.f64(self.rotated) - y) <= S.tolerance_bf16(y, size)).all()


def test_made_behind_other_work_called_on_another_stream(kvc, cuda):
    w, side = Work(kvc, cuda, 31), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    made = w.make()
    torch.cuda.synchronize()                     # (the norms and frequencies are the caller's)
    torch.cuda._sleep(CYCLES)
    w.call(made, stream=side)
    for op in made[:3]:
        op.result(side)
    side.synchronize()
    w.check()
    torch.cuda.synchronize()
    w.case.check(w.got)


@pytest.mark.parametrize("explicit", [True, False])
def test_dropped_while_a_call_is_queued(kvc, cuda, explicit):
    """The memory of an object that is dropped before its call has run, its
    norms and frequencies among it, goes to nobody else until it has."""
    w, side = Work(kvc, cuda, 32), torch.cuda.Stream()
    made = w.make()
    torch.cuda.synchronize()
    sizes = [o.workspace.numel() for o in made[:3]] + [256, 256, 512]
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    with torch.cuda.stream(None if explicit else side):
        w.call(made, **(dict(stream=side) if explicit else {}))
    del made
    other = [torch.full((n,), 255, dtype=torch.uint8, device=cuda) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    w.check()
    assert all(bool((t == 255).all()) for t in other)


def test_made_within_a_capture(kvc, cuda):
    c = Case([7, 3, 12], 9000, True, 3, 33)
    args = c.args(cuda)
    kvc.DraftVerifier(3, 9000, 22)(**args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v = kvc.DraftVerifier(3, 9000, 22)
        got = v(**args)
    for _ in range(3):
        got[2].fill_(7)
        graph.replay()
        v.result()
        c.check(got)
        torch.cuda.synchronize()

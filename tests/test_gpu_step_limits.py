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


def test_two_graphs_of_one_object(kvc, cuda):
    """Captured calls that share an object's workspace, replayed in turn with
    eager calls of it between."""
    for draft, wide in ((True, 0), (True, 3), (False, 3)):
        cases = [Case([7, 3, 12], 9000, draft, wide, 40 + i) for i in range(2)]
        v = kvc.DraftVerifier(3, 9000, 22)
        args, graphs = [c.args(cuda) for c in cases], []
        outs = [v(**a) for a in args]
        torch.cuda.synchronize()
        for a, o in zip(args, outs):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                v(**a, kept=o[0], kept_lens=o[1], out_tokens=o[2])
            graphs.append(graph)
        for turn in range(6):
            i = turn % 2
            for t in outs[i]:
                t.fill_(-7)
            graphs[i].replay()
            if turn % 3 == 0:
                cases[1 - i].check(v(**args[1 - i]))
            v.result()
            cases[i].check(outs[i])


def test_captured_forks_and_releases(kvc, cuda):
    """A graph that forks and one that releases, replayed with new lists,
    padding among them, and an eager call between."""
    lens = np.array([40, 33, 0, 0, 0, 0, 0])
    c = Cache(kvc, cuda, [3, 3, 0, 0, 0, 0, 0], 16, 2, 2, 64, "bf16", 50)
    s = c.share()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
    parents, children, ends, length = i32([0, 0, 0, 0]), i32([-1] * 4), i32([-1] * 4), i32(lens.tolist())
    s.fork(parents, children, length)
    s.release(ends)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        s.fork(parents, children, length)
    with torch.cuda.graph(graphs[1]):
        s.release(ends)
    for who, what, gone in (([0, 1, 0, 0], [2, 3, -1, 4], [3, -1, 2, -1]), ([1, 4, 0, 4], [-1, 2, 3, 5], [4, 5, -1, 3]),
                            ([1, 1, 1, 1], [3, 4, 5, 6], [6, 5, 4, 3])):
        for p, x in zip(who, what):
            lens[x] = lens[p] if x >= 0 else lens[x]
        parents.copy_(i32(who))
        children.copy_(i32(what))
        length.copy_(i32(lens.tolist()))
        graphs[0].replay()
        s.result()
        c.table, c.held, c.count, c.extra = S.fork(c.pools.numpy(), c.table, c.held, c.free, c.count, c.extra, 16, who, what, lens)
        c.same()
        ends.copy_(i32(gone))
        graphs[1].replay()
        s.result()
        c.held, c.free, c.count, c.extra = S.release(c.table, c.held, c.free, c.count, c.extra, gone)
        c.same()
        for x in gone:
            lens[x] = 0 if x >= 0 else lens[x]
    c.release([2, 0, 1])
    assert c.count == c.num_pages and not c.extra.any()


def test_outcomes_of_other_workspaces(kvc, cuda):
    """An outcome is read from a workspace that a call of its own kind has
    written, and from no other."""
    w = Work(kvc, cuda, 60)
    made = w.make()
    for op in made[:3]:
        with pytest.raises(kvc.KvcError):
            op.result()                          # (none has been called)
    w.call(made)
    for op in made[:3]:
        op.result()
    calls = [kvc._lib_verify_result, kvc._lib_compact_result, kvc._lib_shared_result, kvc._lib_attention_result,
             lambda ws, s: kvc._lib_block_table_result(ws, s, None)]
    stream = torch.cuda.current_stream().cuda_stream
    for i, op in enumerate(made[:3]):
        for k, call in enumerate(calls):
            assert call(op.workspace.data_ptr(), stream) == (kvc.KVC_OK if i == k else kvc.KVC_ERR_INVALID)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kvc, cuda, kind):
    """Keys, values and an unfilled page at the far end of pools of more than
    4 GiB: as in near ones."""
    dtype, page, heads, d = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn, 16, 2, 128
    raw = torch.int16 if kind == "bf16" else torch.uint8
    num_pages = (5 << 30) // (page * heads * d * (2 if kind == "bf16" else 1))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
    n = 23
    q, k, v = (torch.randn((n, m, d), device=cuda).to(torch.bfloat16) for m in (4, heads, heads))
    pos = torch.arange(n, device=cuda)
    freq = 100.0 ** (-torch.arange(64, dtype=torch.float64, device=cuda) / 64)
    got = []
    for pages, row, top in ((num_pages, [num_pages - 1, num_pages - 3], num_pages - 2), (4, [3, 1], 2)):
        pools = [torch.empty((pages, page, heads, d), dtype=dtype, device=cuda) for _ in range(2)]
        table = i32([row, [-1, -1]])
        paged = kvc.PagedKV(pools, table, page)
        slots = table[0].long()[pos // page] * page + pos % page
        out = kvc.PagedQKV(paged, 4, freq)(0, q, k, v, slots, pos.int())
        free = torch.full((pages,), top, dtype=torch.int32, device=cuda)
        shared = kvc.SharedPages(paged, i32([2, 0]), free, i32([1]), torch.zeros(pages, dtype=torch.int32, device=cuda))
        shared.fork(i32([0]), i32([1]), i32([n, 0]))
        shared.result()
        assert table[1].tolist() == [row[0], top]
        got.append([out] + [p.view(raw)[x, : y].clone() for p in pools for x, y in ((row[0], page), (row[1], n - page), (top, n - page))])
        shared.release(i32([0, 1]))
        shared.result()
        assert shared.free_pages[:3].tolist() == sorted([*row, top])
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(got[0][2], got[0][3]) and torch.equal(got[0][5], got[0][6])

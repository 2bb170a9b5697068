"""Rows moved together in the pages, pages shared by requests and given back:
every integer and every bit of the pools as the plain forms have them."""
import sys

import numpy as np
import pytest
import torch

import step_reference as S

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dev(x, cuda):
    return torch.from_numpy(np.ascontiguousarray(x)).to(cuda)


class Cache:
    """Pools on the host (as bits) and on the device, and a batch's pages."""

    def __init__(self, kvc, cuda, held, page, layers, heads, d, kind, seed, spare=20, cols=None):
        self.rng = np.random.default_rng(seed)
        self.kvc, self.cuda, self.page = kvc, cuda, page
        self.held = np.array(held, np.int32)
        batch, used = len(held), int(self.held.sum())
        self.num_pages = used + spare
        perm = self.rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((batch, cols or int(self.held.max()) + 3), -7, np.int32)
        at = 0
        for b in range(batch):
            self.table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        self.free, self.count = np.full(self.num_pages, -9, np.int32), spare
        self.free[:spare] = perm[used:]
        self.extra = np.zeros(self.num_pages, np.int32)
        dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        shape = (2 * layers, self.num_pages, page, heads, d)
        bits = torch.int16 if kind == "bf16" else torch.uint8
        self.pools = torch.from_numpy(self.rng.integers(0, 1 << (15 if kind == "bf16" else 8), shape)).to(bits)
        self.on_device = self.pools.to(cuda).view(dtype)
        self.t_table = dev(self.table, cuda)
        self.paged = kvc.PagedKV(list(self.on_device.unbind(0)), self.t_table, page)

    def same_pools(self):
        assert torch.equal(self.on_device.view(self.pools.dtype).cpu(), self.pools)

    def share(self, apart=False):
        c = self.cuda
        self.state = dev(self.held, c), dev(self.free, c), dev(np.array([self.count], np.int32), c), dev(self.extra, c)
        out = (torch.full_like(self.state[0], -5), torch.full_like(self.state[2], -5)) if apart else (None, None)
        self.shared = self.kvc.SharedPages(self.paged, *self.state, held_out=out[0], free_count_out=out[1])
        return self.shared

    def fork(self, parents, children, lens, stream=None):
        self.shared.fork(dev(np.array(parents, np.int32), self.cuda), dev(np.array(children, np.int32), self.cuda),
                         dev(np.array(lens, np.int32), self.cuda))
        self.shared.result()
        self.table, self.held, self.count, self.extra = S.fork(self.pools.numpy(), self.table, self.held, self.free, self.count,
                                                               self.extra, self.page, parents, children, lens)
        self.same()

    def release(self, requests):
        self.shared.release(dev(np.array(requests, np.int32), self.cuda))
        self.shared.result()
        self.held, self.free, self.count, self.extra = S.release(self.table, self.held, self.free, self.count, self.extra,
                                                                 requests)
        self.same()

    def same(self):
        s = self.shared
        for name, got, want in (("table", self.t_table, self.table), ("held", s.held_out, self.held),
                                ("free", s.free_pages, self.free), ("count", s.free_count_out, [self.count]),
                                ("extra", s.extra, self.extra)):
            assert np.array_equal(got.cpu().numpy(), want), name
        self.same_pools()


# ---------------------------------------------------------------- compaction

def paths(nodes, rng, most=12):
    kept, lens = [], []
    for n in nodes:
        a = int(rng.integers(0, min(n, most) + 1))
        path = np.sort(rng.choice(n, a, replace=False)) if a else np.zeros(0, np.int64)
        kept.append(np.concatenate([path, np.full(n - a, -1)]))
        lens.append(a)
    return (np.concatenate(kept).astype(np.int32) if len(nodes) else np.zeros(0, np.int32)), np.array(lens, np.int32)


@pytest.mark.parametrize("page,layers,heads,d,kind", [(1, 1, 1, 64, "e4m3"), (16, 3, 8, 128, "bf16"), (5, 2, 3, 192, "bf16"),
                                                      (24, 1, 2, 256, "e4m3"), (64, 5, 1, 64, "bf16")])
@pytest.mark.parametrize("most", [1, 12, 300])
def test_compact(kvc, cuda, page, layers, heads, d, kind, most):
    say(f"compact page {page} layers {layers} heads {heads} d {d} {kind} most {most}")
    rng = np.random.default_rng(page + most)
    nodes = np.array([most, 1, 0, most // 2, 3 if most > 3 else 1, most])
    context = rng.integers(0, 40, 6)
    context[1], context[5] = 0, page - 1
    c = Cache(kvc, cuda, (-(-(context + nodes) // page)).tolist(), page, layers, heads, d, kind, page)
    kept, lens = paths(nodes, rng, most)
    if most > 12:                                # long moves: every second row; all but the first; none
        kept[:300], lens[0] = np.concatenate([np.arange(0, 300, 2), np.full(150, -1)]), 150
        kept[-300:], lens[5] = np.concatenate([np.arange(1, 300), [-1]]), 299
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    op = kvc.PagedCompaction(c.paged)
    op(dev(starts, cuda), dev(context.astype(np.int32), cuda), dev(kept, cuda), dev(lens, cuda))
    op.result()
    S.compact(c.pools.numpy(), c.table, page, starts, context, kept, lens)
    c.same_pools()


def test_compact_without_context_and_of_nothing(kvc, cuda):
    c = Cache(kvc, cuda, [2, 1], 8, 2, 1, 64, "bf16", 3)
    op = kvc.PagedCompaction(c.paged)
    starts, kept, lens = np.array([0, 10, 14], np.int32), np.full(20, -1, np.int32), np.array([3, 4], np.int32)
    kept[:3], kept[10:14] = [2, 5, 9], range(4)
    op(dev(starts, cuda), None, dev(kept, cuda), dev(lens, cuda))
    op.result()
    S.compact(c.pools.numpy(), c.table, 8, starts, [0, 0], kept, lens)
    c.same_pools()
    op(dev(np.zeros(3, np.int32), cuda), None, dev(np.zeros(0, np.int32), cuda), dev(np.zeros(2, np.int32), cuda))
    op.result()
    c.same_pools()


def test_compact_of_what_does_not_fit(kvc, cuda):
    """The bad sequence is reported and left as it was, the others are moved."""
    def refused(bad, starts=(0, 6, 12, 18), context=(3, 9, 14), kept=None, lens=(3, 3, 3), table=None, moved=(0, 1, 2)):
        c = Cache(kvc, cuda, [3, 3, 3], 8, 2, 1, 64, "bf16", 4, cols=3)
        if table is not None:
            c.t_table[table[0], table[1]] = table[2]
        k = np.tile([0, 3, 5, -1, -1, -1], 3).astype(np.int32)
        for i, x in (kept or {}).items():
            k[i] = x
        op = kvc.PagedCompaction(c.paged)
        op(*(dev(np.array(x, np.int32), cuda) for x in (starts, context, k, lens)))
        with pytest.raises(kvc.KvcError) as e:
            op.result()
        assert e.value.status == kvc.KVC_ERR_INVALID
        keep = np.array([lens[b] if b in moved else 0 for b in range(3)])
        S.compact(c.pools.numpy(), c.table, 8, np.arange(4) * 6, context, k, keep)
        c.same_pools()

    refused(0, lens=(7, 3, 3), moved=(1, 2))
    refused(1, lens=(3, -1, 3), moved=(0, 2))
    refused(0, context=(-1, 9, 14), moved=(1, 2))
    refused(2, context=(3, 9, 19), moved=(0, 1))               # 25 tokens of 24
    refused(2, context=(3, 9, 0x7FFFFFFF), moved=(0, 1))
    refused(1, kept={7: 0}, moved=(0, 2))
    refused(1, kept={8: 6}, moved=(0, 2))
    refused(1, kept={6: -2}, moved=(0, 2))
    refused(2, starts=(0, 6, 12, 19), moved=(0, 1))
    refused(2, starts=(0, 6, 12, 11), moved=(0, 1))
    refused(1, table=(1, 1, 99), moved=(0, 2))                 # positions 9 to 14 of it lie there
    refused(1, table=(1, 1, -1), moved=(0, 2))


def test_compact_past_32_bits(kvc, cuda):
    """Rows at the far end of pools of more than 4 GiB."""
    page, heads, d = 16, 8, 128
    num_pages = (5 << 30) // (page * heads * d * 2)
    pools = [torch.zeros((num_pages, page, heads, d), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    table = torch.tensor([[num_pages - 1, num_pages - 3]], dtype=torch.int32, device=cuda)
    rows = torch.randn((20, heads, d), device=cuda).to(torch.bfloat16)
    paged = kvc.PagedKV(pools, table, page)
    pos = torch.arange(20, device=cuda)
    kvc.kvc_paged_append(paged, 0, rows, -rows, table[0].long()[pos // page] * page + pos % page)
    op = kvc.PagedCompaction(paged)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
    op(i32([0, 18]), i32([2]), i32([0, 5, 17] + [-1] * 15), i32([3]))
    op.result()
    assert torch.equal(pools[0][-1, 2:5], rows[[2, 7, 19]]) and torch.equal(pools[1][-1, 2:5], -rows[[2, 7, 19]])


# ---------------------------------------------------------------- forks and releases

@pytest.mark.parametrize("page,layers,heads,d,kind", [(1, 1, 1, 64, "e4m3"), (16, 3, 8, 128, "bf16"), (5, 2, 3, 192, "bf16"),
                                                      (24, 1, 2, 256, "e4m3"), (64, 5, 1, 64, "bf16")])
@pytest.mark.parametrize("apart", [False, True])
def test_fork_and_release(kvc, cuda, page, layers, heads, d, kind, apart):
    say(f"fork page {page} layers {layers} heads {heads} d {d} {kind} apart {apart}")
    lens = np.array([3 * page + page // 2, 0, 2 * page, page - 1, 0, 0, 0, 0, 0, 0])
    held = [-(-int(n) // page) + (1 if i == 0 else 0) for i, n in enumerate(lens)]
    c = Cache(kvc, cuda, held, page, layers, heads, d, kind, page)
    c.share(apart)
    c.fork([0, 2, 0, 3, 5, 1], [4, 5, -1, 6, -1, 7], lens)
    if apart:
        return
    lens[[4, 5, 6]] = lens[[0, 2, 3]]
    c.fork([4, 5, 0], [8, 9, 1], lens)           # a fork of a fork
    c.release([0, -1, 9])
    c.release([2, 5, 8])
    c.release([])
    c.release([4, 6, 3, 1, 7, 0])
    assert not c.held.any() and not c.extra.any() and c.count == c.num_pages


@pytest.mark.parametrize("seed", range(3))
def test_many_requests(kvc, cuda, seed):
    """Hundreds of requests in long rows, released in batches."""
    rng = np.random.default_rng(seed)
    parents, each, page = 40, 20, 4
    lens = np.zeros(parents * (each + 1), np.int64)
    lens[:parents] = rng.integers(0, 6000, parents)
    held = [-(-int(n) // page) for n in lens]
    c = Cache(kvc, cuda, held, page, 1, 1, 64, "e4m3", seed, spare=parents * each + 50)
    c.share()
    children = parents + rng.permutation(parents * each)
    c.fork(np.repeat(np.arange(parents), each), children, lens)
    order = rng.permutation(len(lens))
    for part in np.array_split(order, 3):
        c.release(part)
    assert not c.held.any() and not c.extra.any() and c.count == c.num_pages


def test_as_many_as_a_call_takes(kvc, cuda):
    page = 16
    lens = np.zeros(1025, np.int64)
    lens[0] = 35
    c = Cache(kvc, cuda, [3] + [0] * 1024, page, 1, 1, 64, "bf16", 8, spare=1024)
    c.share()
    c.fork(np.zeros(1024, np.int64), np.arange(1024, 0, -1), lens)
    assert c.count == 0
    c.release(np.arange(1, 1025))
    c.release([0])
    with pytest.raises(kvc.KvcError):
        c.shared.release(torch.zeros(1025, dtype=torch.int32, device=cuda))


def test_forks_that_do_not_fit_change_nothing(kvc, cuda):
    page, lens = 16, np.array([40, 20, 0, 0, 0])

    def refused(status, parents, children, lens=lens, spare=20, free=None, change=None):
        c = Cache(kvc, cuda, [3, 2, 0, 0, 0], page, 2, 1, 64, "bf16", 5, spare=spare)
        s = c.share()
        if free is not None:
            s.free_pages[spare - 1] = free
            c.free[spare - 1] = free
        if change:
            change(c)
        s.fork(*(dev(np.array(x, np.int32), cuda) for x in (parents, children, lens)))
        with pytest.raises(kvc.KvcError) as e:
            s.result()
        assert e.value.status == status
        c.same()
        return c

    inv = kvc.KVC_ERR_INVALID
    refused(inv, [0, 0], [2, 2])
    refused(inv, [0, 1], [2, 0])                 # the child holds pages
    refused(inv, [0], [5])
    refused(inv, [0], [-2])
    refused(inv, [5], [2])
    refused(inv, [-1], [2])
    refused(inv, [2], [2])
    refused(inv, [0], [2], lens=np.array([49, 20, 0, 0, 0]))   # more tokens than its pages hold
    refused(inv, [0], [2], lens=np.array([-1, 20, 0, 0, 0]))
    refused(inv, [3], [2], lens=np.array([40, 20, 0, 1, 0]))
    refused(kvc.KVC_ERR_CAPACITY, [0, 1, 1], [2, 3, 4], spare=2)
    refused(inv, [0], [2], free=99)
    refused(inv, [0], [2], free=-1)

    def height(x):
        def change(c):
            c.shared.free_count.fill_(x)
            c.count = x
        return change
    refused(inv, [0], [2], change=height(-1))
    refused(inv, [0], [2], change=height(26))

    def last_page(c):                            # that the parent's last tokens would be copied from
        c.table[0, 2] = 77
        c.t_table[0, 2] = 77
    refused(inv, [0], [2], change=last_page)

    def held(c):
        c.held[0] = 1 << 20
        c.shared.held.fill_(0)
        c.shared.held.copy_(dev(c.held, cuda))
    refused(inv, [0], [2], change=held)
    c = refused(inv, [0, 0], [2, 2])
    c.fork([0], [2], lens)                       # and the next one is sound
    # a page number outside the pools among the shared ones: entered, not counted
    c = Cache(kvc, cuda, [3, 2, 0, 0, 0], page, 2, 1, 64, "bf16", 6)
    c.table[0, 1] = 1000
    c.t_table[0, 1] = 1000
    s = c.share()
    s.fork(*(dev(np.array(x, np.int32), cuda) for x in ([0], [2], lens)))
    with pytest.raises(kvc.KvcError):
        s.result()
    assert c.t_table[2, :2].tolist() == [c.table[0, 0], 1000] and int(s.extra.sum()) == 1


def test_releases_that_do_not_fit(kvc, cuda):
    def run(requests, change=None, spare=20):
        c = Cache(kvc, cuda, [3, 2, 4, 0, 0], 16, 1, 1, 64, "bf16", 7, spare=spare)
        c.share()
        if change:
            change(c)
            c.t_table.copy_(dev(c.table, cuda))
            c.shared.extra.copy_(dev(c.extra, cuda))
        c.shared.release(dev(np.array(requests, np.int32), cuda))
        with pytest.raises(kvc.KvcError) as e:
            c.shared.result()
        return c, e.value.status

    inv = kvc.KVC_ERR_INVALID
    for requests, sound in (([0, 1, 0], [0, 1]), ([0, 5], [0]), ([-2, 0], [0])):
        c, status = run(requests)
        assert status == inv
        c.held, c.free, c.count, c.extra = S.release(c.table, c.held, c.free, c.count, c.extra, sound)
        c.same()
    # a page in two requests that was never counted twice: given back once
    def twice(c):
        c.table[1, 0] = c.table[0, 0]
    c, status = run([0, 1], twice)
    pages = sorted(set(c.table[0, :3]) | set(c.table[1, :2]))
    assert status == inv and c.shared.free_pages[20:20 + len(pages)].tolist() == pages
    assert int(c.shared.free_count) == 20 + len(pages) and not c.shared.extra.any()
    # a page number outside the pools is passed over
    def outside(c):
        c.table[0, 1], c.table[2, 3] = -1, c.num_pages
    c, status = run([0, 2], outside)
    pages = sorted([c.table[0, 0], c.table[0, 2], *c.table[2, :3]])
    assert status == inv and c.shared.free_pages[20:25].tolist() == pages and int(c.shared.free_count) == 25
    assert c.shared.held_out.tolist() == [0, 2, 0, 0, 0]
    # a height of the stack that cannot be
    for x in (-1, 30):
        c, status = run([0], lambda c: c.shared.free_count.fill_(x))
        c.count = x
        assert status == inv
        c.same()
    # held counts that cannot be
    for x in (-1, 8):
        def held(c):
            c.held[0] = x
            c.shared.held.copy_(dev(c.held, cuda))
        c, status = run([0, 1], held)
        assert status == inv
        c.held, c.free, c.count, c.extra = S.release(c.table, c.held, c.free, c.count, c.extra, [1])
        c.same()
    # more pages than the stack has room for: what fits is pushed, and the next call is sound
    c, status = run([0, 2], lambda c: c.shared.free_count.fill_(26))
    pages = sorted([*c.table[0, :3], *c.table[2, :4]])
    assert status == kvc.KVC_ERR_CAPACITY and c.shared.free_pages[26:29].tolist() == pages[:3]
    assert int(c.shared.free_count) == 29
    c.shared.free_count.fill_(0)
    c.shared.release(dev(np.array([1], np.int32), cuda))
    c.shared.result()
    assert c.shared.free_pages[:2].tolist() == sorted(c.table[1, :2])


def test_refusals(kvc, cuda):
    c = Cache(kvc, cuda, [3, 2], 16, 1, 1, 64, "bf16", 9)
    s = c.share()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
    for parents, children, lens in ((i32([0]).long(), i32([1]), i32([1, 1])), (i32([0, 1]), i32([1]), i32([1, 1])),
                                    (i32([0]), i32([1]), i32([1])), (i32([0]), i32([1]).cpu(), i32([1, 1]))):
        with pytest.raises(ValueError):
            s.fork(parents, children, lens)
    with pytest.raises(ValueError):
        s.release(torch.zeros(3, device=cuda))
    held, free, count, extra = c.state
    for bad in (dict(held=held[:1]), dict(free_pages=free[:-1]), dict(free_count=held), dict(extra=extra[:-1]),
                dict(extra=extra.long()), dict(held_out=count), dict(free_count_out=held)):
        with pytest.raises(ValueError):
            kvc.SharedPages(c.paged, **{**dict(held=held, free_pages=free, free_count=count, extra=extra), **bad})
    op = kvc.PagedCompaction(c.paged)
    ok = [i32([0, 1, 2]), i32([0, 0]), i32([0, 0]), i32([1, 1])]
    for i, bad in ((0, i32([0, 1])), (1, i32([0])), (2, i32([0, 0]).long()), (3, i32([0])), (2, i32([0, 0]).cpu())):
        with pytest.raises(ValueError):
            op(*ok[:i], bad, *ok[i + 1:])

"""Block tables, slot maps and appends on the GPU against the plain forms:
every integer equal, every row of the pool its exact or correctly rounded
value, other rows untouched."""
import sys

import numpy as np
import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dev(x, cuda):
    return torch.from_numpy(np.ascontiguousarray(x)).to(cuda)


class State:
    """A batch's pages on the host and on the device."""

    def __init__(self, kvc, cuda, batch, page, max_pages, num_pages, held, max_rows, seed, apart=False):
        rng = np.random.default_rng(seed)
        perm = rng.permutation(num_pages).astype(np.int32)
        self.table = np.full((batch, max_pages), -7, np.int32)
        at = 0
        for b in range(batch):
            self.table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        self.held, self.page, self.max_rows = np.array(held, np.int32), page, max_rows
        self.free = np.full(num_pages, -9, np.int32)
        self.count = num_pages - at
        self.free[:self.count] = perm[at:]
        i32 = dict(dtype=torch.int32, device=cuda)
        out = (torch.full((batch,), -5, **i32), torch.full((1,), -5, **i32)) if apart else (None, None)
        self.t = kvc.BlockTable(dev(self.table, cuda), dev(self.held, cuda), dev(self.free, cuda),
                                dev(np.array([self.count], np.int32), cuda), page, num_pages,
                                torch.full((batch + 1,), -5, **i32),
                                torch.full((max_rows,), -5, dtype=torch.int64, device=cuda),
                                torch.full((max_rows,), -5, **i32), held_out=out[0], free_count_out=out[1])
        self.cuda = cuda

    def step(self, cached, new, trim):
        args = [None if x is None else dev(np.array(x, np.int32), self.cuda) for x in (cached, new)]
        zero = np.zeros(len(self.held), np.int32)
        want = R.block_table(self.table, self.held, self.free, self.count, self.page,
                             zero if cached is None else cached, zero if new is None else new, self.max_rows, trim)
        self.t(*args, trim=trim)
        assert self.t.result() == want[4][-1]
        self.table, self.held, self.free, self.count = want[:4]
        for name, got, exp in zip(("table", "held", "free", "count", "row_starts", "slots", "positions"),
                                  (self.t.block_table, self.t.held_out, self.t.free_pages, self.t.free_count_out,
                                   self.t.row_starts, self.t.slots, self.t.positions),
                                  (want[0], want[1], want[2], np.array([want[3]], np.int32), *want[4:])):
            assert np.array_equal(got.cpu().numpy(), exp), name


@pytest.mark.parametrize("batch,page,longest,new,max_rows", [
    (1, 1, 5, 3, 8), (1, 16, 64, 1, 1), (3, 16, 100, 20, 64), (8, 24, 400, 64, 600),
    (65, 7, 50, 9, 700), (1025, 5, 12, 3, 4000), (40, 16, 2000, 700, 30000), (1500, 16, 100, 40, 70000),
])
@pytest.mark.parametrize("apart", [False, True])
def test_steps_of_a_batch(kvc, cuda, batch, page, longest, new, max_rows, apart):
    say(f"batch {batch} page {page} longest {longest} new {new} max_rows {max_rows} apart {apart}")
    rng = np.random.default_rng(batch * 131 + page)
    cap = -(-longest // page) + 2
    cached = rng.integers(0, longest - new + 1, batch)
    held = np.minimum(-(-cached // page) + rng.integers(0, 2, batch), cap)
    fresh = rng.integers(0, new + 1, batch)
    fresh[0] = new
    while fresh.sum() > max_rows:
        fresh //= 2
    s = State(kvc, cuda, batch, page, cap, int(held.sum()) + batch * cap + 3, held, max_rows, batch, apart)
    s.step(cached, fresh, False)
    if apart:
        return
    total = cached + fresh
    # a trim to what was accepted, some requests finished; then the finished rows start anew
    kept = np.maximum(total - rng.integers(0, new + 1, batch), 0)
    kept[rng.random(batch) < 0.3] = 0
    s.step(kept, None, True)
    s.step(None if not kept.any() else kept, np.minimum(fresh, longest - kept), True)
    s.step(None, np.zeros(batch, np.int64), False)


@pytest.mark.parametrize("batch,max_rows", [(40, 200), (40, 3000), (1100, 9000)])
@pytest.mark.parametrize("fresh", [False, True])
def test_requests_that_come_with_tokens_and_no_pages(kvc, cuda, batch, max_rows, fresh):
    """A cache that was decoded elsewhere, or a prefix to be filled: pages for
    the cached tokens are taken along with those of the new ones, whole pages,
    page borders and single tokens among them."""
    rng = np.random.default_rng(batch + fresh)
    cached = rng.integers(0, 200, batch)
    cached[:8] = [0, 1, 15, 16, 17, 32, 160, 199]
    held = np.minimum(rng.integers(0, 3, batch) * rng.integers(0, 2, batch), -(-cached // 16))
    new = rng.integers(0, 6, batch) if fresh else np.zeros(batch, np.int64)
    if fresh:
        new[:8] = [0, 15, 1, 0, 15, 16, 2, 40]
    s = State(kvc, cuda, batch, 16, 16, 16 * batch, held, max_rows, 9)
    s.step(cached, new if fresh else None, False)
    s.step(cached, None, True)


@pytest.mark.parametrize("batch", [5, 1100])
def test_without_slots_or_positions(kvc, cuda, batch):
    """The maps are left out singly or both: the table and the row starts are
    the same, and without them no number of rows is too large."""
    i32 = dict(dtype=torch.int32, device=cuda)
    got = []
    for slots, positions in ((True, True), (True, False), (False, True), (False, False)):
        t = kvc.BlockTable(torch.full((batch, 8), -1, **i32), torch.zeros(batch, **i32),
                           torch.arange(8 * batch, **i32), torch.full((1,), 8 * batch, **i32), 16, 8 * batch,
                           torch.zeros(batch + 1, **i32),
                           torch.zeros(128 * batch, dtype=torch.int64, device=cuda) if slots else None,
                           torch.zeros(128 * batch, **i32) if positions else None)
        new = torch.arange(batch, **i32) % 129
        t(None, new)
        assert t.result() == int(new.sum())
        got.append((t.block_table, t.row_starts, t.held, t.free_count))
    for g in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], g))


def test_trim_undoes_a_step(kvc, cuda):
    s = State(kvc, cuda, 5, 16, 10, 64, [1, 0, 2, 3, 1], 200, 3)
    before, count = s.free.copy(), s.count
    cached = np.array([16, 0, 20, 40, 3])
    s.step(cached, np.array([30, 16, 0, 64, 1]), False)
    s.step(cached, None, True)
    assert s.count == count and np.array_equal(s.free[:count], before[:count])


def test_failed_steps_leave_the_state(kvc, cuda):
    def refused(status, cached, new, held=(1, 2), rows=64, free=None, trim=False, count=None):
        s = State(kvc, cuda, 2, 16, 4, 8, list(held), rows, 1)
        if free is not None:
            s.t.free_pages[:] = free
        if count is not None:
            s.t.free_count.fill_(count)
        keep = [x.clone() for x in (s.t.block_table, s.t.held, s.t.free_pages, s.t.free_count)]
        s.t(*[dev(np.array(x, np.int32), cuda) for x in (cached, new)], trim=trim)
        with pytest.raises(kvc.KvcError) as e:
            s.t.result()
        assert e.value.status == status
        if free is None:
            for was, now in zip(keep, (s.t.block_table, s.t.held, s.t.free_pages, s.t.free_count)):
                assert torch.equal(was, now)
            assert not s.t.row_starts.any() and (s.t.slots == -1).all() and (s.t.positions == -1).all()
        return s

    inv, cap = kvc.KVC_ERR_INVALID, kvc.KVC_ERR_CAPACITY
    refused(inv, [-1, 5], [2, 2])
    refused(inv, [5, 5], [2, -2])
    refused(inv, [5, 5], [2, 2], count=9)
    refused(inv, [5, 5], [2, 2], count=-1)
    refused(cap, [5, 64], [2, 1])                                # more pages than the row has columns
    refused(cap, [0x7FFFFFFF, 5], [0x7FFFFFFF, 1])
    refused(cap, [60, 60], [4, 4], count=3)                      # five pages wanted, three free
    refused(cap, [5, 5], [40, 30])                               # more rows than the maps hold
    s = State(kvc, cuda, 2, 16, 4, 8, [1, 2], 64, 1)
    s.t.held[1] = 5
    s.t(None, None)
    with pytest.raises(kvc.KvcError):
        s.t.result()
    # a page number outside the pools: its rows get no slot, the others do
    s = refused(inv, [14, 30], [4, 4], free=99)
    slots = s.t.slots.cpu().numpy()
    assert (slots[[2, 3, 6, 7]] == -1).all() and (slots[[0, 1, 4, 5]] >= 0).all()


@pytest.mark.parametrize("src,pool,strided", [("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "e4m3", True),
                                              ("bf16", "e4m3", False), ("e4m3", "e4m3", True), ("e4m3", "e4m3", False)])
@pytest.mark.parametrize("rows,heads,d,page", [(1, 1, 64, 1), (3, 8, 128, 16), (77, 3, 192, 5), (1000, 2, 256, 24),
                                               (513, 16, 64, 64)])
def test_append(kvc, cuda, src, pool, strided, rows, heads, d, page):
    say(f"append {src} -> {pool} strided {strided} rows {rows} heads {heads} d {d} page {page}")
    g = torch.Generator(device="cpu").manual_seed(rows * 7 + d)
    kind = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
    num_pages = -(-rows // page) + 2

    def values(shape, t):
        # magnitudes from below the smallest e4m3 step to beyond its largest value
        x = torch.randn(shape, generator=g) * torch.exp2(torch.empty(shape).uniform_(-12, 11, generator=g))
        x = x.to(kind[t])
        flat = x.view(torch.int16 if t == "bf16" else torch.uint8).view(-1)
        odd = [0x7FC0, 0x7F80, -128, -32768, 0, 1] if t == "bf16" else [0x7F, 0xFF, 0x80, 0x7E, 0xFE, 1]
        flat[: len(odd)] = torch.tensor(odd, dtype=torch.int32).to(flat.dtype)
        return x

    pools = [values((4, num_pages, page, heads, d), pool)[:2][i].clone().to(cuda) for i in range(2)]
    layers = [p.clone() for p in pools] + pools                  # layer 0 stays, layer 1 gets the rows
    keep = [p.clone() for p in layers]
    wide = values((rows, 3 * heads, d), src).to(cuda)
    k, v = (wide[:, :heads], wide[:, 2 * heads:]) if strided else (wide[:, :heads].contiguous(), wide[:, heads:2 * heads].contiguous())
    slots = torch.randperm(num_pages * page, generator=g)[:rows]
    if rows > 2:
        slots[1], slots[rows // 2] = -1, num_pages * page        # no slot; one past the pools
    scale = (0.75, 3.0) if src != pool else (1.0, 1.0)
    paged = kvc.PagedKV(layers, torch.zeros((1, 1), dtype=torch.int32, device=cuda), page)
    kvc.kvc_paged_append(paged, 1, k, v, slots.to(cuda), *scale)
    torch.cuda.synchronize()
    bits = torch.int16 if pool == "bf16" else torch.uint8
    for i, (x, c) in enumerate(((k, scale[0]), (v, scale[1]))):
        assert torch.equal(layers[i].view(bits), keep[i].view(bits))
        want = keep[2 + i].view(bits).view(-1, heads, d).clone()
        there = (slots >= 0) & (slots < num_pages * page)
        y = x[there.to(cuda)]
        if src != pool:
            y = (y.float() / c).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = layers[2 + i].view(bits).view(-1, heads, d)
        want[slots[there].to(cuda)] = y.contiguous().view(bits)
        if src != pool:                                          # a NaN's sign is not kept track of
            nan = (want & 0x7F) == 0x7F
            assert torch.equal((got & 0x7F) == 0x7F, nan)
            want, got = want.masked_fill(nan, 0x7F), got.masked_fill(nan, 0x7F)
        assert torch.equal(got, want)


def test_append_of_no_rows(kvc, cuda):
    pools = [torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    paged = kvc.PagedKV(pools, torch.zeros((1, 1), dtype=torch.int32, device=cuda), 16)
    none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=cuda)
    kvc.kvc_paged_append(paged, 0, none, none, torch.empty(0, dtype=torch.int64, device=cuda))
    torch.cuda.synchronize()
    assert not pools[0].any() and not pools[1].any()

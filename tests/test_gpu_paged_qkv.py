"""Norms, rotation and append in one pass, against float64: every query and
key within the roundings counted in step_reference, values as the append
writes them, other rows untouched."""
import sys

import numpy as np
import pytest
import torch

import step_reference as S

pytestmark = pytest.mark.gpu

KIND = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.uint8)


class Case:
    def __init__(self, kvc, cuda, rows, q_heads, heads, d, page, pool, rotary, interleaved, norm, strided, seed,
                 positions=None, layers=2, far=1 << 17):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.kvc, self.cuda, self.pool, self.interleaved, self.page = kvc, cuda, pool, interleaved, page
        self.heads, self.q_heads, self.d, self.rows, self.layers = heads, q_heads, d, rows, layers
        num_pages = -(-rows // page) + 2
        self.pools = [torch.randn((num_pages, page, heads, d), generator=g).to(KIND[pool]).to(cuda) for _ in range(2 * layers)]
        wide = torch.randn((rows, q_heads + 2 * heads, d), generator=g)
        wide = (wide * torch.exp(torch.randn(d, generator=g))).to(torch.bfloat16).to(cuda)
        parts = wide[:, :q_heads], wide[:, q_heads:q_heads + heads], wide[:, q_heads + heads:]
        self.q, self.k, self.v = parts if strided else [t.contiguous() for t in parts]
        self.slots = torch.randperm(num_pages * page, generator=g)[:rows]
        self.positions = torch.randint(0, far, (rows,), generator=g, dtype=torch.int32)
        if rows > 3:
            self.slots[1], self.slots[rows // 2], self.positions[2] = -1, num_pages * page, -1
            self.positions[0], self.positions[3] = 0, 0x7FFFFFFF
        if rows > 5:
            self.slots[4], self.positions[4] = -1, -5
        if positions is not None:
            self.positions = positions
        dtype = torch.float32 if norm == "f32" else torch.bfloat16
        weights = (1 + 0.3 * torch.randn((2, layers, d), generator=g)).to(dtype).to(cuda)
        self.q_norm = weights[0] if norm in ("bf16", "f32", "q") else None
        self.k_norm = weights[1] if norm in ("bf16", "f32", "k") else None
        self.freq = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(rotary // 2, 1))
        self.scale = (0.07, 0.3) if pool == "e4m3" else (1.0, 1.0)
        self.eps = 1e-5
        self.paged = kvc.PagedKV(self.pools, torch.zeros((1, 1), dtype=torch.int32, device=cuda), page)

    def op(self):
        return self.kvc.PagedQKV(self.paged, self.q_heads, self.freq.to(self.cuda) if len(self.freq) else None, self.q_norm,
                                 self.k_norm, eps=self.eps, interleaved=self.interleaved, k_scale=self.scale[0],
                                 v_scale=self.scale[1])

    def check(self, layer, out, keep_out, keep_pools, q=None):
        pos = self.positions.numpy()
        real = pos >= 0
        freq = self.freq.numpy()
        y, size = S.norm_rotate(S.f64(self.q if q is None else q), None if self.q_norm is None else S.f64(self.q_norm[layer]),
                                self.eps, pos, freq, self.interleaved)
        got = S.f64(out)
        assert (np.abs(got - y) <= S.tolerance_bf16(y, size))[real].all()
        assert torch.equal(bits(out)[~torch.from_numpy(real)], bits(keep_out)[~torch.from_numpy(real)])
        n_slots = self.pools[0].shape[0] * self.page
        there = real & ((self.slots >= 0) & (self.slots < n_slots)).numpy()
        y, size = S.norm_rotate(S.f64(self.k), None if self.k_norm is None else S.f64(self.k_norm[layer]), self.eps, pos, freq,
                                self.interleaved)
        at = self.slots.numpy()[there]
        for i, (now, was) in enumerate(zip(self.pools, keep_pools)):
            flat, old = bits(now).view(-1, self.heads, self.d), bits(was).view(-1, self.heads, self.d)
            other = torch.ones(n_slots, dtype=torch.bool)
            if i // 2 == layer:
                other[at] = False
            assert torch.equal(flat[other], old[other])
        got = S.f64(self.pools[2 * layer].view(-1, self.heads, self.d)[torch.from_numpy(at)])
        if self.pool == "bf16":
            ok = np.abs(got - y[there]) <= S.tolerance_bf16(y, size)[there]
        else:
            z = y / self.scale[0]
            ok = np.abs(got - np.clip(z[there], -448, 448)) <= S.tolerance_e4m3(z, size / self.scale[0])[there]
        assert ok.all()
        # the values: what the append writes
        plain = [p.clone() for p in keep_pools]
        paged = self.kvc.PagedKV(plain, torch.zeros((1, 1), dtype=torch.int32, device=self.cuda), self.page)
        slots = torch.where(self.positions >= 0, self.slots, -1).to(self.cuda)
        self.kvc.kvc_paged_append(paged, layer, self.v, self.v, slots, k_scale=self.scale[0], v_scale=self.scale[1])
        assert torch.equal(bits(self.pools[2 * layer + 1]), bits(plain[2 * layer + 1]))

    def run(self, layer=1, op=None, **kw):
        keep = [p.clone() for p in self.pools]
        out = torch.full((self.rows, self.q_heads, self.d), 3.0, dtype=torch.bfloat16, device=self.cuda)
        keep_out = out.clone()
        op = op or self.op()
        got = op(layer, self.q, self.k, self.v, self.slots.to(self.cuda), self.positions.to(self.cuda), out=out, **kw)
        assert got is out
        torch.cuda.synchronize()
        self.check(layer, out, keep_out, keep)


@pytest.mark.parametrize("rows,q_heads,heads,d,page", [
    (1, 1, 1, 64, 1), (2, 32, 8, 128, 16), (7, 5, 1, 192, 5), (33, 12, 3, 256, 24), (130, 3, 3, 64, 16), (1111, 16, 2, 128, 16),
])
@pytest.mark.parametrize("pool,interleaved,norm,strided", [
    ("bf16", False, "bf16", True), ("bf16", True, "f32", False), ("e4m3", False, "f32", True), ("e4m3", True, "bf16", False),
])
def test_every_head_shape(kvc, cuda, rows, q_heads, heads, d, page, pool, interleaved, norm, strided):
    for rotary in sorted({d, d // 2 if d % 32 == 0 else 16, 16, 0}):
        say(f"rows {rows} q {q_heads} kv {heads} d {d} rotary {rotary} {pool} interleaved {interleaved} norm {norm}")
        Case(kvc, cuda, rows, q_heads, heads, d, page, pool, rotary, interleaved, norm, strided, rows + d).run()


@pytest.mark.parametrize("norm", ["q", "k", None])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norms_left_out(kvc, cuda, norm, interleaved):
    for rotary in (128, 48):
        Case(kvc, cuda, 19, 8, 2, 128, 16, "bf16", rotary, interleaved, norm, True, 5).run(0)


@pytest.mark.parametrize("rows", [1000, 3000])
def test_many_rows(kvc, cuda, rows):
    """Rows to a wave each, all their heads."""
    Case(kvc, cuda, rows, 32, 8, 128, 16, "bf16", 128, False, "bf16", True, 6).run()
    Case(kvc, cuda, rows, 7, 1, 192, 16, "e4m3", 96, True, "f32", True, 7).run()


def test_far_positions(kvc, cuda):
    """Every position is as exact as a near one."""
    Case(kvc, cuda, 300, 4, 1, 128, 16, "bf16", 128, False, "bf16", True, 8, far=0x7FFFFFFF).run()


def test_queries_in_place_and_no_queries(kvc, cuda):
    c = Case(kvc, cuda, 40, 8, 2, 128, 16, "bf16", 128, False, "bf16", True, 9)
    keep, before = [p.clone() for p in c.pools], c.q.clone()
    out = c.op()(0, c.q, c.k, c.v, c.slots.to(cuda), c.positions.to(cuda), out=c.q)
    assert out is c.q
    c.check(0, out, before, keep, q=before)
    c = Case(kvc, cuda, 40, 0, 2, 128, 16, "bf16", 128, False, "bf16", True, 10)
    c.run()
    c = Case(kvc, cuda, 0, 8, 2, 128, 16, "bf16", 128, False, "bf16", False, 11)
    c.run()


def test_without_positions(kvc, cuda):
    c = Case(kvc, cuda, 9, 8, 2, 128, 16, "bf16", 0, False, "bf16", True, 12, positions=torch.zeros(9, dtype=torch.int32))
    keep = [p.clone() for p in c.pools]
    out = c.op()(1, c.q, c.k, c.v, c.slots.to(cuda))
    c.check(1, out, out, keep)


def test_values_beyond_the_squares_of_float32(kvc, cuda):
    """Heads whose squares pass float32 are normed all the same; an infinity or
    a NaN stays in its head; tiny heads are ruled by eps."""
    c = Case(kvc, cuda, 24, 8, 2, 128, 16, "bf16", 0, False, "bf16", False, 13)
    c.q[4:8] *= 1e25
    c.q[8:10] = 3e38
    c.k[5] *= -1e24
    c.q[11] *= 1e-30
    c.q[12] = 0
    c.run()
    q, k = c.q.clone(), c.k.clone()
    c.q[13, 1, 7], c.q[13, 3, 100], c.k[14, 0, 5], c.v[14, 1, 3], c.v[15, 0, 9] = np.inf, np.nan, -np.inf, np.nan, np.inf
    op = c.op()
    out = op(0, c.q, c.k, c.v, c.slots.to(cuda), c.positions.to(cuda)).float().cpu()
    clean = op(0, q, k, c.v, c.slots.to(cuda), c.positions.to(cuda)).float().cpu()
    real = (c.positions >= 0)
    hit = torch.zeros((24, 8), dtype=torch.bool)
    hit[13, 1] = hit[13, 3] = True
    hit[~real] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[13, 1, 7].isnan() and (out[13, 1, :7] == 0).all() and out[13, 3].isnan().all()


def test_values_of_bf16_pages_keep_every_bit(kvc, cuda):
    """All 65536 patterns of bf16, NaN and infinities among them, as values."""
    rows = 512
    c = Case(kvc, cuda, rows, 1, 1, 128, 16, "bf16", 128, False, "bf16", False, 14)
    c.v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(rows, 1, 128).to(cuda)
    slots = torch.arange(rows, device=cuda)
    c.op()(0, c.q, c.k, c.v, slots, torch.zeros(rows, dtype=torch.int32, device=cuda))
    assert torch.equal(bits(c.pools[1]).view(-1, 1, 128)[:rows], bits(c.v))


@pytest.mark.parametrize("scale", [1.0, 0.07, 3.0, 1e-30, 1e30, 2.0 ** -126, 3e38, 1e-42, 448.0, 1.0 / 3.0])
def test_values_of_e4m3_pages_are_the_appends(kvc, cuda, scale):
    """... and rounded to an e4m3 cache, for every pattern, as the append
    rounds them, to the bit (a NaN's sign aside)."""
    rows = 512
    c = Case(kvc, cuda, rows, 1, 1, 128, 16, "e4m3", 0, False, None, False, 14)
    c.v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(rows, 1, 128).to(cuda)
    slots = torch.arange(rows, device=cuda)
    plain = [p.clone() for p in c.pools]
    kvc.PagedQKV(c.paged, 1, k_scale=scale, v_scale=scale)(0, c.q, c.v, c.v, slots)
    kvc.kvc_paged_append(kvc.PagedKV(plain, c.paged.block_table, 16), 0, c.v, c.v, slots, k_scale=scale, v_scale=scale)
    for x, y in zip(c.pools, plain):
        x, y = bits(x), bits(y)
        nan = (y & 0x7F) == 0x7F
        assert torch.equal((x & 0x7F) == 0x7F, nan) and torch.equal(x[~nan], y[~nan])


def test_more_rows_than_a_launch_has_waves(kvc, cuda):
    """Waves that take several rows: as the rows by themselves."""
    rows = 150001
    q, k, v = (torch.randn((rows, n, 64), device=cuda).to(torch.bfloat16) for n in (5, 1, 1))
    pos = torch.randint(-1, 5000, (rows,), device=cuda, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=cuda) / 32)
    slots = torch.randperm(rows + 15, device=cuda)[:rows]
    got = []
    for step in (rows, 1 << 14):
        pools = [torch.zeros((-(-(rows + 15) // 16), 16, 1, 64), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
        op = kvc.PagedQKV(kvc.PagedKV(pools, torch.zeros((1, 1), dtype=torch.int32, device=cuda), 16), 5, freq)
        out = torch.zeros_like(q)
        for i in range(0, rows, step):
            op(0, q[i:i + step], k[i:i + step], v[i:i + step], slots[i:i + step], pos[i:i + step], out=out[i:i + step])
        got.append((out, *pools))
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_two_streams_and_a_graph(kvc, cuda):
    """Calls on two streams through one object, and a captured one replayed on
    new rows, equal those of the current stream."""
    c = Case(kvc, cuda, 64, 8, 2, 128, 16, "bf16", 128, False, "bf16", True, 15)
    op, slots, pos = c.op(), c.slots.to(cuda), c.positions.to(cuda).clamp(min=0)
    want = op(0, c.q, c.k, c.v, slots, pos).clone()
    keep = [p.clone() for p in c.pools]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [op(i, c.q, c.k, c.v, slots, pos, stream=streams[i]) for i in (0, 1)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(c.pools[0], keep[0]) and torch.equal(c.pools[1], keep[1])
    q, k, v = c.q.contiguous(), c.k.contiguous(), c.v.contiguous()
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(0, q, k, v, slots, pos, out=out)
    for i in range(3):
        for t in (q, k, v):
            t.normal_()
        pos.random_(0, 5000)
        graph.replay()
        replayed = out.clone(), c.pools[0].clone(), c.pools[1].clone()
        eager = op(0, q, k, v, slots, pos)
        assert torch.equal(replayed[0], eager) and torch.equal(replayed[1], c.pools[0]) and torch.equal(replayed[2], c.pools[1])
        torch.cuda.synchronize()


def test_refusals(kvc, cuda):
    c = Case(kvc, cuda, 6, 8, 2, 128, 16, "bf16", 128, False, "bf16", True, 16)
    op, slots, pos = c.op(), c.slots.to(cuda), c.positions.to(cuda)
    ok = dict(q=c.q, k=c.k, v=c.v, slots=slots, positions=pos)
    for bad in (dict(q=c.q.float()), dict(q=c.q[:5]), dict(k=c.q), dict(v=c.v[:, :, :64]), dict(slots=slots.int()),
                dict(slots=slots[:5]), dict(positions=pos.long()), dict(positions=None), dict(q=c.q.cpu()),
                dict(out=torch.empty((6, 128, 8), dtype=torch.bfloat16, device=cuda).transpose(1, 2)),
                dict(k=c.k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            op(0, **{**ok, **bad})
    for layer in (-1, 2):
        with pytest.raises(kvc.KvcError):
            op(layer, **ok)
    f = c.freq.to(cuda)
    for kw in (dict(frequencies=f.float()), dict(frequencies=f[:12]), dict(frequencies=torch.cat([f, f])), dict(eps=0.0),
               dict(eps=float("nan")), dict(k_scale=0.5), dict(q_norm=c.q_norm[0]), dict(q_norm=c.q_norm.float()),
               dict(q_norm=c.q_norm.half(), k_norm=None), dict(q_heads=-1)):
        with pytest.raises(ValueError):
            kvc.PagedQKV(c.paged, **{**dict(q_heads=8, frequencies=f, q_norm=c.q_norm, k_norm=c.k_norm), **kw})

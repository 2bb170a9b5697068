"""Attention over a paged cache on the GPU against float64, at the sizes and
masks where it can go wrong."""
import sys

import numpy as np
import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu

KIND = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


class Case:
    """Pools, table, queries and masks; ref() gives the float64 values."""

    def __init__(self, kvc, cuda, contexts, nodes, heads, ratio, d, kind, page, tree, seed=0, layers=2, layer=1,
                 scale=None, words=None, q_gain=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cpu").manual_seed(seed + 1)
        self.contexts, self.nodes = np.array(contexts), np.array(nodes)
        total = self.contexts + self.nodes
        pages = -(-total // page)
        cols = int(pages.max()) + 1
        num_pages = int(pages.sum()) + 2
        perm = rng.permutation(num_pages)
        self.table = rng.integers(0, num_pages, (len(total), cols)).astype(np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.pools = [torch.randn((num_pages, page, heads, d), generator=g).to(KIND[kind]).to(cuda)
                      for _ in range(2 * layers)]
        self.starts = np.concatenate([[0], np.cumsum(self.nodes)]).astype(np.int32)
        rows = int(self.starts[-1])
        self.q = (q_gain * torch.randn((rows, heads * ratio, d), generator=g)).to(torch.bfloat16).to(cuda)
        self.words = -(-int(self.nodes.max()) // 64) if words is None else words
        self.mask = R.tree(self.nodes, self.words, rng) if tree else None
        self.page, self.d, self.layer, self.scale = page, d, layer, scale
        self.kvc, self.cuda = kvc, cuda
        self.scales = (1.0, 1.0)

    def dev(self, x, dtype=torch.int32):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(self.cuda)

    def paged(self):
        return self.kvc.PagedKV(self.pools, self.dev(self.table), self.page)

    def run(self, hint=0, most=0, q=None, max_rows=None, **kw):
        q = self.q if q is None else q
        att = self.kvc.PagedAttention(self.paged(), q.shape[1], max_rows or q.shape[0], hint, most, self.scale,
                                      *self.scales)
        got = att(self.layer, q, self.dev(self.starts), self.dev(self.contexts), self.dev(self.mask, torch.int64), **kw)
        att.result()
        return got

    def ref(self):
        scale = (self.d ** -0.5 if self.scale is None else self.scale) * self.scales[0]
        return R.attention(R.to_f64(self.pools[2 * self.layer]), R.to_f64(self.pools[2 * self.layer + 1]), self.table,
                           self.page, R.to_f64(self.q), self.starts, self.contexts,
                           None if self.mask is None else self.mask.view(np.uint64), scale, self.scales[1])

    def check(self, got, ref=None):
        out, lse, loose, score = ref or self.ref()
        tol_out, tol_lse = R.tolerances(out, loose, score, int((self.contexts + self.nodes).max()), self.d)
        o, z = R.to_f64(got[0]), R.to_f64(got[1])
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(z), empty)
        assert not o[empty].any()
        bad = np.abs(o - out) > tol_out
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], float((np.abs(o - out) / tol_out).max()))
        off = np.abs(z[~empty] - lse[~empty]) - tol_lse[~empty]
        assert not (off > 0).any(), float(off.max())


SHAPES = [
    # contexts, nodes, heads, ratio, d, page
    ([0], [1], 1, 1, 64, 16),
    ([1], [1], 2, 2, 128, 1),
    ([31, 32, 33, 0, 63], [1, 1, 1, 1, 1], 2, 4, 128, 16),
    ([100, 0, 17], [3, 5, 0], 1, 3, 192, 5),
    ([15, 250, 31], [33, 1, 64], 2, 2, 256, 24),
    ([700, 129], [7, 16], 3, 5, 64, 100),
    ([40, 5], [70, 130], 2, 1, 128, 16),
    ([300], [20], 1, 17, 128, 32),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_float64(kvc, cuda, shape, tree, kind):
    say(f"case {shape} tree {tree} {kind}")
    c = Case(kvc, cuda, *shape[:5], kind, shape[5], tree, seed=shape[4])
    ref = c.ref()
    c.check(c.run(), ref)
    for hint in (1, 64):                                   # other row tiles, the same values
        c.check(c.run(hint=hint), ref)


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("e4m3", 64), ("bf16", 256), ("e4m3", 192)])
@pytest.mark.parametrize("page", [8, 16, 48])
def test_long_contexts_are_split(kvc, cuda, kind, d, page):
    say(f"split {kind} {d} page {page}")
    c = Case(kvc, cuda, [5000, 37, 9001], [2, 9, 1], 2, 4, d, kind, page, True, seed=page)
    ref = c.ref()
    c.check(c.run(), ref)
    # bounds that are too small or too large change the launch alone
    c.check(c.run(most=1), ref)
    c.check(c.run(hint=9, most=1 << 30), ref)


def test_many_sequences(kvc, cuda):
    rng = np.random.default_rng(5)
    contexts, nodes = rng.integers(0, 150, 150), rng.integers(0, 4, 150)
    c = Case(kvc, cuda, contexts, nodes, 2, 2, 64, "bf16", 16, True, seed=6)
    ref = c.ref()
    c.check(c.run(), ref)
    contexts[70] = 6000
    c = Case(kvc, cuda, contexts, nodes + 1, 1, 8, 128, "e4m3", 16, False, seed=7)
    c.check(c.run())


def test_a_piece_of_a_prompt(kvc, cuda):
    c = Case(kvc, cuda, [333, 0], [200, 129], 2, 4, 128, "bf16", 16, False, seed=8)
    c.check(c.run())


def test_peaked_scores_and_scales(kvc, cuda):
    """Scores of hundreds (one token takes all), a scale of its own, and the
    scales of an e4m3 cache."""
    c = Case(kvc, cuda, [500, 90], [4, 12], 2, 3, 128, "e4m3", 16, True, seed=9, scale=0.2, q_gain=8.0)
    c.scales = (0.37, 2.5)
    c.check(c.run())


def test_rows_that_see_nothing(kvc, cuda):
    c = Case(kvc, cuda, [0, 40, 0], [5, 3, 70], 2, 4, 128, "bf16", 16, True, seed=10)
    c.mask[0] = 0                                          # context 0, no drafted token: empty
    c.mask[3] = 0
    c.mask[5] = 0                                          # 40 tokens of context alone
    c.mask[9:11] = 0
    c.mask[20] = [1 << 40, 0]
    ref = c.ref()
    assert np.isneginf(ref[1]).any()
    c.check(c.run(), ref)


def test_bits_behind_the_last_drafted_token_are_ignored(kvc, cuda):
    c = Case(kvc, cuda, [33, 7], [5, 40], 1, 4, 64, "bf16", 16, True, seed=11, words=2)
    ref = c.ref()
    full = c.mask.copy()
    for b in range(2):
        for r in range(c.starts[b], c.starts[b + 1]):
            full[r, 0] |= ~((1 << int(c.nodes[b])) - 1)
            full[r, 1] = -1
    c.mask = full
    c.check(c.run(), ref)
    # fewer words than drafted tokens: those behind them are not seen
    c = Case(kvc, cuda, [33, 7], [5, 100], 1, 4, 64, "bf16", 16, True, seed=12, words=1)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_wild_values_in_masked_places(kvc, cuda, kind, d):
    """NaN and infinities in K and V of drafted tokens reach the rows that see
    them and no others; what stands in a page behind the last token reaches
    none."""
    c = Case(kvc, cuda, [20, 64], [9, 40], 2, 2, d, kind, 16, True, seed=13)
    clean = c.ref()
    heads = 2
    kp, vp = c.pools[2 * c.layer].view(-1, heads, d), c.pools[2 * c.layer + 1].view(-1, heads, d)
    raw = torch.int16 if kind == "bf16" else torch.uint8
    kr, vr = kp.view(raw), vp.view(raw)
    nan = 0x7FC0 if kind == "bf16" else 0x7F
    inf = 0x7F80 if kind == "bf16" else 0x7F               # e4m3 has no infinity
    touched = np.zeros(len(c.q), bool)

    def slot(b, pos):
        return int(c.table[b, pos // 16]) * 16 + pos % 16

    for b in range(2):                                     # the rest of the last page
        total = int(c.contexts[b] + c.nodes[b])
        for pos in range(total, -(-total // 16) * 16):
            kr[slot(b, pos)] = nan
            vr[slot(b, pos)] = nan
    c.check(c.run(), clean)

    vr[slot(0, 20 + 4), 1, 3] = nan
    kr[slot(0, 20 + 6), 0, 5] = nan
    vr[slot(1, 64 + 7), 0] = inf
    vr[slot(1, 64 + 39), 1, d - 1] = inf
    got = c.run()
    o, z = R.to_f64(got[0]), R.to_f64(got[1])
    out, lse, loose, score = clean
    tol_out, tol_lse = R.tolerances(out, loose, score, 104, d)
    bits = c.mask.view(np.uint64)
    for r in range(len(o)):
        b = 0 if r < c.starts[1] else 1
        for a in range(4):
            h = a // 2
            see = lambda j: bool((int(bits[r, 0]) >> j) & 1)
            hit = np.zeros(d, bool)
            lost = False
            if b == 0 and h == 1 and see(4):
                hit[3] = True
            if b == 0 and h == 0 and see(6):
                lost = True                                # a NaN score
            if b == 1 and h == 0 and see(7):
                hit[:] = True
            if b == 1 and h == 1 and see(39):
                hit[d - 1] = True
            if lost:
                assert np.isnan(o[r, a]).all() and np.isnan(z[r, a])
                continue
            touched[r] |= hit.any()
            want = np.isnan if kind == "e4m3" or b == 0 else np.isposinf
            assert want(o[r, a][hit]).all(), (r, a)
            assert (np.abs(o[r, a] - out[r, a])[~hit] <= tol_out[r, a][~hit]).all(), (r, a)
            assert abs(z[r, a] - lse[r, a]) <= tol_lse[r, a]
    assert touched.any()


def test_opposite_infinities_make_nan(kvc, cuda):
    c = Case(kvc, cuda, [0], [3], 1, 1, 64, "bf16", 16, False, seed=14)
    v = c.pools[2 * c.layer + 1].view(-1, 1, 64)
    s0 = int(c.table[0, 0]) * 16
    v[s0 + 1, 0, 0], v[s0 + 2, 0, 0], v[s0 + 2, 0, 1] = float("inf"), float("-inf"), float("-inf")
    o = c.run()[0].float().cpu()
    assert torch.isfinite(o[0]).all()
    assert o[1, 0, 0] == float("inf") and torch.isfinite(o[1, 0, 1:]).all()
    assert torch.isnan(o[2, 0, 0]) and o[2, 0, 1] == float("-inf") and torch.isfinite(o[2, 0, 2:]).all()


def test_strided_queries_and_outputs(kvc, cuda):
    c = Case(kvc, cuda, [77, 300], [6, 3], 2, 4, 128, "bf16", 16, True, seed=15)
    ref = c.ref()
    wide = torch.zeros((len(c.q), 3, 8, 128), dtype=torch.bfloat16, device=cuda)
    wide[:, 1] = c.q
    out = torch.full((len(c.q), 16, 128), 7.0, dtype=torch.bfloat16, device=cuda)
    got = c.run(q=wide[:, 1], out=out[:, 8:])
    c.check(got, ref)
    assert (out[:, :8] == 7).all()
    heads_first = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    c.check(c.run(q=heads_first), ref)


def test_rows_behind_the_last_sequence_stay(kvc, cuda):
    c = Case(kvc, cuda, [50, 20], [2, 4], 2, 2, 64, "bf16", 16, True, seed=16)
    ref = c.ref()
    n = len(c.q)
    pad = torch.cat([c.q, torch.randn((5, 4, 64), device=cuda).to(torch.bfloat16)])
    c.mask = np.concatenate([c.mask, np.full((5, 1), -1, np.int64)])
    out = torch.full((n + 5, 4, 64), 3.0, dtype=torch.bfloat16, device=cuda)
    lse = torch.full((n + 5, 4), 3.0, device=cuda)
    c.run(q=pad, out=out, lse=lse, max_rows=n + 9)
    c.check((out[:n], lse[:n]), ref)
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()


def test_lengths_and_pages_that_do_not_fit_are_reported(kvc, cuda):
    def make():
        return Case(kvc, cuda, [50, 20, 90], [2, 4, 1], 2, 2, 64, "bf16", 16, False, seed=17)

    def refused(c, status=kvc.KVC_ERR_INVALID, rows=None):
        out = torch.full_like(c.q, 3.0)
        with pytest.raises(kvc.KvcError) as e:
            c.run(out=out)
        assert e.value.status == status
        return out

    c = make()
    ref = c.ref()
    c.contexts[0] = -1
    out = refused(c)
    assert (out[:2] == 3).all()                            # that sequence is not written, the others are
    assert np.abs(R.to_f64(out)[2:] - ref[0][2:]).max() < 0.1
    c = make()
    c.contexts[2] = 16 * c.table.shape[1]
    assert (refused(c)[6:] == 3).all()
    c = make()
    c.starts[3] = 8                                        # past the rows
    assert (refused(c)[6:] == 3).all()
    c = make()
    c.starts[:] = [0, 6, 2, 7]                             # falling
    refused(c)
    c = make()
    c.starts[0] = -3
    refused(c)
    for page in (-1, 1 << 30):
        c = make()
        c.table[1, 0] = page
        out = refused(c)
        assert np.abs(R.to_f64(out)[:2] - ref[0][:2]).max() < 0.1
    c = make()
    c.run()                                                # nothing of it stays


def test_no_rows(kvc, cuda):
    c = Case(kvc, cuda, [50, 20], [2, 4], 2, 2, 64, "bf16", 16, False, seed=18)
    c.starts[:] = 0
    att = kvc.PagedAttention(c.paged(), 4, 8)
    out, lse = att(1, c.q[:0], c.dev(c.starts), c.dev(c.contexts))
    att.result()
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_function_form_and_argument_checks(kvc, cuda):
    c = Case(kvc, cuda, [50, 20], [2, 4], 2, 2, 64, "bf16", 16, True, seed=19)
    ref = c.ref()
    args = (c.paged(), c.layer, c.q, c.dev(c.starts), c.dev(c.contexts))
    c.check(kvc.kvc_paged_attention(*args, c.dev(c.mask, torch.int64)), ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kvc.kvc_paged_attention(*args, c.dev(c.mask, torch.int64), stream=s)
    c.check(got, ref)
    att = kvc.PagedAttention(c.paged(), 4, 6)
    good = args[2:]
    for bad in ((c.q.float(), *good[1:]), (c.q[:, :2], *good[1:]), (c.q.cpu(), *good[1:]),
                (torch.cat([c.q, c.q]), *good[1:]), (good[0], good[1].long(), good[2]),
                (good[0], good[1][:2], good[2]), (good[0], good[1], good[2].cpu())):
        with pytest.raises(ValueError):
            att(0, *bad)
    with pytest.raises(ValueError):
        att(0, *good, c.dev(c.mask, torch.int32))
    with pytest.raises(kvc.KvcError):
        att(2, *good)
    with pytest.raises(kvc.KvcError):
        att(-1, *good)
    with pytest.raises(kvc.KvcError):
        kvc.PagedAttention(c.paged(), 5, 6)
    with pytest.raises(kvc.KvcError):
        kvc.PagedAttention(c.paged(), 4, 6, k_scale=0.0)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 4.0])
@pytest.mark.parametrize("nodes", [[1, 2], [20, 9]])
def test_scales(kvc, cuda, scale, nodes):
    """Negative, zero, vanishing and large softmax scales."""
    c = Case(kvc, cuda, [300, 77], nodes, 2, 2, 64, "bf16", 16, True, seed=20, scale=scale)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("gain", [0.02, 0.3, 3.0])
@pytest.mark.parametrize("nodes", [[1, 3], [40, 21]])
def test_scores_that_grow_along_the_sequence(kvc, cuda, kind, gain, nodes):
    """Maxima that are passed by little, at every token, and by much: keys
    that point more and more along (or against) one direction that the
    queries share."""
    c = Case(kvc, cuda, [1500, 200], nodes, 1, 4, 128, kind, 16, False, seed=21, scale=1.0)
    one = torch.zeros(128, device=cuda)
    one[5] = 1.0
    for b in range(2):
        total = int(c.contexts[b] + c.nodes[b])
        t = torch.arange(total, device=cuda)
        slot = torch.from_numpy(c.table[b]).to(cuda).long()[t // 16] * 16 + t % 16
        k = c.pools[2 * c.layer].view(torch.int16 if kind == "bf16" else torch.uint8).view(-1, 1, 128)
        step = (t if b == 0 else total - t).float() * gain / 10
        rows = (step.clamp(max=400)[:, None, None] * one).to(KIND[kind])
        k[slot] = rows.view(k.dtype)
    c.q = (one + 0.01 * c.q.float()).to(torch.bfloat16)
    c.check(c.run())


def test_more_sequences_than_lanes_and_long_ones_among_them(kvc, cuda):
    rng = np.random.default_rng(22)
    contexts, nodes = rng.integers(0, 60, 200), rng.integers(0, 3, 200)
    contexts[[3, 66, 199]], nodes[[3, 66, 199]] = [7000, 3000, 5000], [25, 1, 30]
    c = Case(kvc, cuda, contexts, nodes, 1, 2, 64, "bf16", 16, True, seed=23)
    ref = c.ref()
    c.check(c.run(), ref)
    c.check(c.run(hint=30), ref)


def test_one_row_or_one_head_of_any_stride(kvc, cuda):
    c = Case(kvc, cuda, [20], [1], 1, 1, 64, "bf16", 16, False, seed=24)
    ref = c.ref()
    wide = torch.zeros((1, 3, 67), dtype=torch.bfloat16, device=cuda).as_strided((1, 1, 64), (67, 13, 1))
    wide.copy_(c.q)
    c.check(c.run(q=wide), ref)


def test_masks_without_rows_or_words(kvc, cuda):
    c = Case(kvc, cuda, [20, 3], [2, 1], 1, 1, 64, "bf16", 16, False, seed=25)
    att = kvc.PagedAttention(c.paged(), 1, 3)
    starts, contexts = c.dev(c.starts), c.dev(c.contexts)
    with pytest.raises(ValueError):                        # no words: not the same as no mask
        att(1, c.q, starts, contexts, torch.zeros((3, 0), dtype=torch.int64, device=cuda))
    att(1, c.q[:0], torch.zeros_like(starts), contexts, torch.zeros((0, 1), dtype=torch.int64, device=cuda))
    att.result()


@pytest.mark.parametrize("nodes", [1, 9])
def test_large_batches(kvc, cuda, nodes):
    """More items than workgroups, sequences far behind the first 64, empty
    ones between them; split or an item a workgroup."""
    rng = np.random.default_rng(26)
    batch = 1500
    contexts, rows = rng.integers(0, 40, batch), rng.integers(0, nodes + 1, batch)
    contexts[[0, 700, 1499]], rows[[0, 700, 1499]] = 2000, nodes
    c = Case(kvc, cuda, contexts, rows, 2, 2, 64, "bf16", 16, False, seed=27)
    ref = c.ref()
    for hint in (nodes, 30):
        c.check(c.run(hint=hint), ref)
        c.check(c.run(hint=hint, most=60), ref)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [[3, 2], [70, 40]])
def test_wild_values_of_split_sequences(kvc, cuda, kind, nodes):
    """NaN (and infinities of bf16) in V of drafted tokens where several
    workgroups share a sequence."""
    c = Case(kvc, cuda, [3000, 500], nodes, 2, 4, 128, kind, 16, True, seed=28)
    v = c.pools[2 * c.layer + 1].view(-1, 2, 128)
    for b, j, ch, x in ((0, 1, 5, float("nan")), (0, nodes[0] - 1, 127, float("inf")), (1, 0, 64, float("-inf"))):
        t = int(c.contexts[b]) + j
        v[int(c.table[b, t // 16]) * 16 + t % 16, :, ch] = x
    ref = c.ref()
    got = c.run()
    o, out = R.to_f64(got[0]), np.array(ref[0])
    # an unseen one has weight 0 in the plain form, which leaves it out by rows
    special = ~np.isfinite(out)
    assert special.any() and np.array_equal(np.isnan(o), np.isnan(out))
    assert np.array_equal(o[np.isinf(out)], out[np.isinf(out)])
    tol_out, tol_lse = R.tolerances(np.where(special, 0.0, out), np.where(special, 0.0, ref[2]), ref[3], 3100, 128)
    assert (np.abs(o - out)[~special] <= tol_out[~special]).all()
    assert (np.abs(R.to_f64(got[1]) - ref[1]) <= tol_lse).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 12, 7])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_every_kernel(kvc, cuda, d, page, kind):
    """Each channel count, type and way of finding pages, with few rows, up to
    64 and more a KV head, short and split, trees and chains, over tiles that
    masks cut."""
    for tree in (True, False):
        c = Case(kvc, cuda, [90, 1100, 5], [70, 33, 40], 1, 2, d, kind, page, tree, seed=29)
        ref = c.ref()
        for hint in (1, 20, 70):
            for most in (0, 100):
                c.check(c.run(hint=hint, most=most), ref)

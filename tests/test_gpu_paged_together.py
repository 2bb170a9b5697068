"""The paged cache's calls as a serving step uses them: a compressed prompt
decoded into pages that the block table handed out, drafted tokens appended
and attended to, what was rejected given back; the step captured in a graph
and replayed; calls on several streams; a cache whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import paged_reference as R
from entropy_coding_amd import workloads as W

pytestmark = pytest.mark.gpu

HEADS, RATIO, D, PAGE = 2, 4, 128, 16


def i32(x, cuda):
    return torch.tensor(x, dtype=torch.int32, device=cuda)


class Server:
    """Two sequences on one layer: pools, block table, append and attention."""

    def __init__(self, kvc, cuda, kv_dtype=torch.bfloat16, batch=2, cols=12, num_pages=40, max_rows=32):
        self.kvc, self.cuda = kvc, cuda
        self.pools = [torch.zeros((num_pages, PAGE, HEADS, D), dtype=kv_dtype, device=cuda) for _ in range(2)]
        self.table = torch.full((batch, cols), -1, dtype=torch.int32, device=cuda)
        g = torch.Generator(device="cpu").manual_seed(3)
        self.free = torch.randperm(num_pages, generator=g).to(torch.int32).to(cuda)
        self.count = i32([num_pages], cuda)
        self.held = torch.zeros(batch, dtype=torch.int32, device=cuda)
        self.starts = torch.zeros(batch + 1, dtype=torch.int32, device=cuda)
        self.slots = torch.zeros(max_rows, dtype=torch.int64, device=cuda)
        self.tab = kvc.BlockTable(self.table, self.held, self.free, self.count, PAGE, num_pages, self.starts, self.slots)
        self.paged = kvc.PagedKV(self.pools, self.table, PAGE)
        self.att = kvc.PagedAttention(self.paged, HEADS * RATIO, max_rows, rows_per_sequence=8)

    def draft(self, context, new, k, v, q, mask, out=None, lse=None):
        self.tab(context, new)
        self.kvc.kvc_paged_append(self.paged, 0, k, v, self.slots[: k.shape[0]])
        return self.att(0, q, self.starts, context, mask, out=out, lse=lse)


def check(server, got, q, starts, contexts, mask, rows):
    out, lse, loose, score = R.attention(R.to_f64(server.pools[0]), R.to_f64(server.pools[1]),
                                         server.table.cpu().numpy(), PAGE, R.to_f64(q[:rows]), starts, contexts,
                                         mask.view(np.uint64), D ** -0.5, 1.0)
    tol_out, tol_lse = R.tolerances(out, loose, score, 400, D)
    assert (np.abs(R.to_f64(got[0][:rows]) - out) <= tol_out).all()
    assert (np.abs(R.to_f64(got[1][:rows]) - lse) <= tol_lse).all()


@pytest.mark.parametrize("kv_dtype", [O.BF16, O.E4M3])
def test_decode_draft_verify(kvc, cuda, kv_dtype):
    """A prompt's stream is decoded into the pages, two steps of drafted trees
    run over it, the rejected part is trimmed, and the pages all come back."""
    tokens, batch = 45, 2
    planes = 2 * batch * HEADS
    kv, mu, sig, samples = W.tiny_case(23, planes, tokens, D, kv_dtype)
    kv_bits = kv.view(torch.int16) if kv_dtype == O.BF16 else kv
    if kv_dtype == O.BF16:                       # planted infinities would make every score NaN
        kv = torch.nan_to_num(kv.float(), nan=0.5, posinf=1.0, neginf=-1.0).clamp(-8, 8).to(torch.bfloat16)
        kv_bits = kv.view(torch.int16)
    else:
        kv_bits = torch.where((kv & 0x7F) == 0x7F, torch.full_like(kv, 0x38), kv)
    mu_d, sig_d = mu.to(cuda), sig.to(cuda)
    prefix = kvc.kvc_build_marginal(samples.to(cuda))
    stream = kvc.kvc_encode(kv_bits.to(cuda), mu_d, sig_d, prefix, (9500, 300), 16)

    s = Server(kvc, cuda, torch.bfloat16 if kv_dtype == O.BF16 else torch.float8_e4m3fn)
    s.tab(i32([tokens] * batch, cuda))           # pages for the prompt, no new rows
    assert s.tab.result() == 0
    ws = torch.empty(kvc.DECODE_WORKSPACE_BYTES, dtype=torch.uint8, device=cuda)
    assert kvc.kvc_decode_paged(stream, mu_d, sig_d, prefix, s.paged, ws) == kvc.KVC_OK
    raw = torch.int16 if kv_dtype == O.BF16 else torch.uint8
    table = s.table.long()
    for p in range(2):
        seq = s.pools[p].view(raw)[table[:, :3]].reshape(batch, 48, HEADS, D)[:, :tokens].permute(0, 2, 1, 3)
        assert torch.equal(seq.reshape(-1, tokens, D).cpu(), kv_bits[p * batch * HEADS:(p + 1) * batch * HEADS])

    rng = np.random.default_rng(1)
    context = np.array([tokens, tokens])
    for step in range(2):
        new = np.array([9, 4]) if step == 0 else np.array([3, 12])
        rows = int(new.sum())
        g = torch.Generator(device="cpu").manual_seed(step)
        qkv = torch.randn((rows, HEADS * (RATIO + 2), D), generator=g).to(torch.bfloat16).to(cuda)
        q, k, v = qkv[:, :HEADS * RATIO], qkv[:, HEADS * RATIO:HEADS * (RATIO + 1)], qkv[:, HEADS * (RATIO + 1):]
        mask = R.tree(new, 1, rng)
        got = s.draft(i32(context.tolist(), cuda), i32(new.tolist(), cuda), k, v, q, torch.from_numpy(mask).to(cuda))
        assert s.tab.result() == rows
        s.att.result()
        check(s, got, q, np.concatenate([[0], np.cumsum(new)]), context, mask, rows)
        context = context + np.array([2, 4])     # what the target accepted
        s.tab(i32(context.tolist(), cuda), trim=True)
        assert s.tab.result() == 0
        assert s.held.tolist() == [-(-int(c) // PAGE) for c in context]
    s.tab(trim=True)                             # both finish
    s.tab.result()
    assert s.count.item() == 40 and sorted(s.free.tolist()) == list(range(40)) and not s.held.any()


def test_a_captured_step(kvc, cuda):
    """Table, append and attention captured once and replayed with new
    lengths, values and masks, eager work and synchronizations between the
    replays; a step that does not fit attends to nothing and leaves the
    state."""
    s, e = Server(kvc, cuda), Server(kvc, cuda)
    n = 24                                       # rows of the captured step, some of them padding
    context, new = i32([0, 0], cuda), i32([0, 0], cuda)
    q = torch.zeros((n, HEADS * RATIO, D), dtype=torch.bfloat16, device=cuda)
    k, v = (torch.zeros((n, HEADS, D), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    mask = torch.zeros((n, 1), dtype=torch.int64, device=cuda)
    out, lse = torch.zeros_like(q), torch.zeros((n, HEADS * RATIO), device=cuda)
    s.draft(context, new, k, v, q, mask, out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.draft(context, new, k, v, q, mask, out, lse)
    rng = np.random.default_rng(2)
    at = np.array([0, 0])
    for step, add in enumerate([[20, 3], [1, 1], [8, 16], [24, 0], [0, 0], [7, 9]]):
        add = np.array(add)
        rows = int(add.sum())
        g = torch.Generator(device="cpu").manual_seed(10 + step)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        m = np.full((n, 1), -1, np.int64)
        m[:rows] = R.tree(add, 1, rng)
        mask.copy_(torch.from_numpy(m))
        context.copy_(i32(at.tolist(), cuda))
        new.copy_(i32(add.tolist(), cuda))
        out.fill_(5.0)
        lse.fill_(5.0)
        graph.replay()
        assert s.tab.result() == rows
        s.att.result()
        got = e.draft(i32(at.tolist(), cuda), i32(add.tolist(), cuda), k, v, q, mask,
                      torch.full_like(q, 5.0), torch.full_like(lse, 5.0))
        assert e.tab.result() == rows
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
        assert (out[rows:] == 5).all() and (lse[rows:] == 5).all()
        assert torch.equal(s.table, e.table) and torch.equal(s.pools[0], e.pools[0]) and torch.equal(s.held, e.held)
        if rows:
            check(s, (out, lse), q, np.concatenate([[0], np.cumsum(add)]), at, m[:rows], rows)
        at = at + add
    new.copy_(i32([25, 0], cuda))                # the table has room for them, queries and outputs do not
    out.fill_(5.0)
    graph.replay()
    assert s.tab.result() == 25
    with pytest.raises(kvc.KvcError):
        s.att.result()
    assert (out == 5).all()
    pools = [p.clone() for p in s.pools]
    new.copy_(i32([33, 0], cuda))                # more rows than the table has room for
    graph.replay()
    with pytest.raises(kvc.KvcError):
        s.tab.result()
    s.att.result()
    assert (out == 5).all() and torch.equal(s.pools[0], pools[0]) and torch.equal(s.pools[1], pools[1])
    new.copy_(i32([1, 2], cuda))                 # and the next one is sound again
    context.copy_(i32(at.tolist(), cuda))
    graph.replay()
    assert s.tab.result() == 3
    s.att.result()


def test_calls_on_two_streams(kvc, cuda):
    """Attention objects of their own run at the same time on two streams, on
    tensors made on a third; results equal those of a single stream."""
    contexts, nodes = [3000, 1500, 40], [6, 2, 5]
    from test_gpu_paged_attention import Case
    c = Case(kvc, cuda, contexts, nodes, 2, 4, 128, "bf16", 16, True, seed=40)
    c.check(c.run())
    args = (c.q, c.dev(c.starts), c.dev(c.contexts), c.dev(c.mask, torch.int64))
    want = [kvc.kvc_paged_attention(c.paged(), layer, *args) for layer in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    atts = [kvc.PagedAttention(c.paged(), 8, len(c.q)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [atts[i](i, *args, stream=streams[i]) for i in range(2)]
        for i in range(2):
            atts[i].result(streams[i])
        for w, x in zip(want, got):
            assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    k = torch.randn((7, 2, 128), device=cuda).to(torch.bfloat16)
    slots = torch.arange(7, device=cuda)
    torch.cuda.synchronize()
    kvc.kvc_paged_append(c.paged(), 0, k, k, slots, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(c.pools[0].view(-1, 2, 128)[:7], k)


def test_results_do_not_change_from_call_to_call(kvc, cuda):
    from test_gpu_paged_attention import Case
    for nodes, kind in (([1, 1], "e4m3"), ([30, 11], "bf16")):
        c = Case(kvc, cuda, [4000, 700], nodes, 2, 4, 128, kind, 16, True, seed=41)
        first = c.run()
        for _ in range(3):
            again = c.run()
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_an_object_takes_fewer_rows(kvc, cuda):
    from test_gpu_paged_attention import Case
    big = Case(kvc, cuda, [900, 5000, 10], [20, 30, 40], 2, 2, 64, "bf16", 16, True, seed=42)
    att = kvc.PagedAttention(big.paged(), 4, 90)
    for keep in ([20, 30, 40], [1, 1, 1], [0, 7, 0], [20, 0, 2]):
        rows = np.concatenate([np.arange(big.starts[b], big.starts[b] + keep[b]) for b in range(3)])
        starts = np.concatenate([[0], np.cumsum(keep)]).astype(np.int32)
        mask = big.mask[rows]
        q = big.q[torch.from_numpy(rows).to(cuda)]
        got = att(1, q, big.dev(starts), big.dev(big.contexts), big.dev(mask, torch.int64))
        att.result()
        out, lse, loose, score = R.attention(R.to_f64(big.pools[2]), R.to_f64(big.pools[3]), big.table, 16, R.to_f64(q),
                                             starts, big.contexts, mask.view(np.uint64), 64 ** -0.5, 1.0)
        tol_out, tol_lse = R.tolerances(out, loose, score, 5100, 64)
        assert (np.abs(R.to_f64(got[0]) - out) <= tol_out).all() and (np.abs(R.to_f64(got[1]) - lse) <= tol_lse).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_that_pass_32_bits(kvc, cuda, kind):
    """Pages at the far end of pools of more than 4 GiB."""
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    size = 2 if kind == "bf16" else 1
    num_pages = (5 << 30) // (PAGE * HEADS * D * size)
    pools = [torch.empty((num_pages, PAGE, HEADS, D), dtype=dtype, device=cuda) for _ in range(2)]
    table = torch.tensor([[num_pages - 1, 3, num_pages - 2, num_pages // 2 + 7]], dtype=torch.int32, device=cuda)
    g = torch.Generator(device="cpu").manual_seed(1)
    n = 60
    k, v = (torch.randn((n, HEADS, D), generator=g).to(dtype).to(cuda) for _ in range(2))
    q = torch.randn((n, HEADS * RATIO, D), generator=g).to(torch.bfloat16).to(cuda)
    pos = torch.arange(n, device=cuda)
    slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    paged = kvc.PagedKV(pools, table, PAGE)
    kvc.kvc_paged_append(paged, 0, k, v, slots)
    near = kvc.PagedKV([torch.zeros((4, PAGE, HEADS, D), dtype=dtype, device=cuda) for _ in range(2)],
                       torch.arange(4, dtype=torch.int32, device=cuda)[None], PAGE)
    kvc.kvc_paged_append(near, 0, k, v, pos)
    for rows in (n, 1):                          # both kernels
        starts = i32([0, rows], cuda)
        got, want = (kvc.kvc_paged_attention(p, 0, q[:rows], starts, i32([n - rows], cuda)) for p in (paged, near))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

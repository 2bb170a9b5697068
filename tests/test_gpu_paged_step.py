"""A speculative serving step as a program makes it, all of its calls
together: pages for the new nodes, norms, rotation and append, attention under
the tree's mask, verification, kept rows moved together, pages given back;
eager and captured in a graph, with requests forked and released between the
steps."""
import numpy as np
import pytest
import torch

import paged_reference as R
import step_reference as S

pytestmark = pytest.mark.gpu

HEADS, RATIO, D, PAGE, LAYERS, VOCAB = 2, 4, 128, 16, 2, 300
BATCH, ROWS, PAGES, COLS = 5, 40, 60, 14


class Server:
    def __init__(self, kvc, cuda, kind):
        self.kvc, self.cuda = kvc, cuda
        i32 = dict(dtype=torch.int32, device=cuda)
        g = torch.Generator(device="cpu").manual_seed(2)
        self.pools = [torch.zeros((PAGES, PAGE, HEADS, D), dtype=kind, device=cuda) for _ in range(2 * LAYERS)]
        self.table = torch.full((BATCH, COLS), -1, **i32)
        self.held, self.extra = torch.zeros(BATCH, **i32), torch.zeros(PAGES, **i32)
        self.free, self.count = torch.randperm(PAGES, generator=g).to(torch.int32).to(cuda), torch.full((1,), PAGES, **i32)
        self.starts, self.slots = torch.zeros(BATCH + 1, **i32), torch.zeros(ROWS, dtype=torch.int64, device=cuda)
        self.context = torch.zeros(BATCH, **i32)
        self.scale = dict(k_scale=0.05, v_scale=0.03) if kind == torch.float8_e4m3fn else {}
        self.paged = kvc.PagedKV(self.pools, self.table, PAGE)
        self.tab = kvc.BlockTable(self.table, self.held, self.free, self.count, PAGE, PAGES, self.starts, self.slots)
        norms = (1 + 0.2 * torch.randn((2, LAYERS, D), generator=g)).to(torch.bfloat16).to(cuda)
        freq = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(cuda)
        self.norms, self.freq = norms, freq
        self.qkv = kvc.PagedQKV(self.paged, HEADS * RATIO, freq, norms[0], norms[1], **self.scale)
        self.att = kvc.PagedAttention(self.paged, HEADS * RATIO, ROWS, rows_per_sequence=8, **self.scale)
        self.verify = kvc.DraftVerifier(BATCH, VOCAB, ROWS)
        self.compact = kvc.PagedCompaction(self.paged)
        self.shared = kvc.SharedPages(self.paged, self.held, self.free, self.count, self.extra)
        # a step's inputs and outputs
        z = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device=cuda)
        self.inputs = dict(new=z(BATCH), tokens=z(ROWS), parents=z(ROWS), positions=z(ROWS), mask=z(ROWS, 1, dtype=torch.int64),
                           rows=z(LAYERS, ROWS, HEADS * (RATIO + 2), D, dtype=torch.bfloat16),
                           target=z(ROWS, VOCAB, dtype=torch.float32), draft=z(ROWS, VOCAB, dtype=torch.float32),
                           accept=z(ROWS, dtype=torch.float32), sample=z(BATCH, dtype=torch.float32))
        self.q, self.out = (z(LAYERS, ROWS, HEADS * RATIO, D, dtype=torch.bfloat16) for _ in range(2))
        self.lse = z(LAYERS, ROWS, HEADS * RATIO, dtype=torch.float32)
        self.kept, self.kept_lens, self.out_tokens = z(ROWS), z(BATCH), z(ROWS)

    def step(self):
        i = self.inputs
        self.tab(self.context, i["new"])
        for layer in range(LAYERS):
            q, k, v = i["rows"][layer].split([HEADS * RATIO, HEADS, HEADS], 1)
            self.qkv(layer, q, k, v, self.slots, i["positions"], out=self.q[layer])
            self.att(layer, self.q[layer], self.starts, self.context, i["mask"], out=self.out[layer], lse=self.lse[layer])
        self.verify(i["target"], i["tokens"], self.starts, i["accept"], i["sample"], parents=i["parents"], draft=i["draft"],
                    kept=self.kept, kept_lens=self.kept_lens, out_tokens=self.out_tokens)
        self.compact(self.starts, self.context, self.kept, self.kept_lens)
        self.context.add_(self.kept_lens)
        self.tab(self.context, None, trim=True)

    def results(self):
        for op in (self.att, self.verify, self.compact):
            op.result()
        assert self.tab.result() == 0

    def state(self):
        return (*self.pools, self.table, self.held, self.free[: int(self.count)], self.count, self.context, self.extra)


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def step_inputs(new, context, rng):
    """Host arrays of a step: trees, their masks, positions by depth, rows behind the last sequence as padding."""
    rows = int(sum(new))
    parents, mask, positions = np.zeros(ROWS, np.int32), np.zeros((ROWS, 1), np.int64), np.full(ROWS, -1, np.int32)
    at = 0
    for b, n in enumerate(new):
        depth = np.zeros(n, int)
        for i in range(n):
            up = int(rng.integers(max(0, i - 3), i)) if i else -1
            parents[at + i] = up
            depth[i] = depth[up] + 1 if i else 0
            mask[at + i] = (mask[at + up] if i else 0) | (1 << i)
            positions[at + i] = context[b] + depth[i]
        at += n
    x = 2 * rng.standard_normal((ROWS, VOCAB))
    target, draft = softmax(x), softmax(x + 0.6 * rng.standard_normal((ROWS, VOCAB)))
    tokens = np.zeros(ROWS, np.int32)
    at = 0
    for n in new:
        for i in range(1, n):
            law = draft[at + parents[at + i]].astype(np.float64)
            tokens[at + i] = rng.choice(VOCAB, p=law / law.sum())
        at += n
    return rows, dict(new=np.array(new, np.int32), tokens=tokens, parents=parents, positions=positions, mask=mask,
                      rows=rng.standard_normal((LAYERS, ROWS, HEADS * (RATIO + 2), D)).astype(np.float32), target=target,
                      draft=draft, accept=rng.random(ROWS, dtype=np.float32), sample=rng.random(BATCH, dtype=np.float32))


def rows_at(server, pool, b, n):
    """The first n tokens of request b in a pool, as bits."""
    raw = server.pools[pool].view(torch.int16 if server.pools[pool].element_size() == 2 else torch.uint8)
    pages = server.table[b].long().cpu()[: -(-n // PAGE)]
    return raw[pages.to(raw.device)].reshape(-1, HEADS, D)[:n].cpu()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(kvc, cuda, kind, captured):
    s, plain = Server(kvc, cuda, kind), Server(kvc, cuda, kind)
    rng = np.random.default_rng(3)
    graph = None
    if captured:
        s.step()                                 # (of nothing)
        s.results()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
    have = {b: [torch.zeros((0, HEADS, D)) for _ in range(2 * LAYERS)] for b in range(BATCH)}   # rows that requests keep
    events = {2: ("fork", [0, 0], [3, 4]), 5: ("release", [1, 3]), 6: ("fork", [4, 0], [1, 3]), 9: ("release", [0, 1, 2, 3, 4])}
    for turn in range(10):
        if turn in events:
            what, *who = events[turn]
            for x in (s, plain):
                lists = [torch.tensor(w, dtype=torch.int32, device=cuda) for w in who]
                if what == "fork":
                    x.shared.fork(*lists, x.context)
                    x.context[lists[1].long()] = x.context[lists[0].long()]
                else:
                    x.shared.release(*lists)
                    x.context[lists[0].long()] = 0
                x.shared.result()
            if what == "fork":
                for p, c in zip(*who):
                    have[c] = list(have[p])
            else:
                for r in who[0]:
                    have[r] = [t[:0] for t in have[r]]
        context = plain.context.cpu().numpy().copy()
        live = context > 0 if turn not in (0, 9) else np.array([turn == 0] * 3 + [False] * 2)
        most = 13 if turn == 0 else 8
        new = [int(rng.integers(1, most)) if live[b] else 0 for b in range(BATCH)]
        rows, host = step_inputs(new, context, rng)
        for x in (s, plain):
            for name, t in x.inputs.items():
                t.copy_(torch.from_numpy(host[name]))
            x.out.fill_(5)
            x.q.fill_(5)
        graph.replay() if captured else s.step()
        s.results()
        plain.step()
        plain.results()
        for x, y in zip(s.state(), plain.state()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        for name in ("q", "out", "lse", "kept", "kept_lens", "out_tokens"):
            x, y = getattr(s, name), getattr(plain, name)
            n = rows if name != "kept_lens" else BATCH
            assert torch.equal(x[:n], y[:n]) if name in ("kept", "kept_lens", "out_tokens") else torch.equal(x[:, :n], y[:, :n])
        assert (s.q[:, rows:] == 5).all() and (s.out[:, rows:] == 5).all()
        # what was kept, by the plain walk
        starts = np.concatenate([[0], np.cumsum(new)])
        walked = S.verify(starts, host["tokens"], host["parents"], host["target"], host["draft"], host["accept"], host["sample"])
        kept = s.kept.cpu().numpy()
        for b, (path, tokens) in enumerate(walked):
            at = int(starts[b])
            assert kept[at:at + len(path)].tolist() == path
            assert s.out_tokens.cpu().numpy()[at:at + len(tokens)].tolist() == tokens
            assert int(s.context[b]) == context[b] + len(path)
        # each request's rows: those it had, and its kept nodes' in their order
        wide = torch.from_numpy(host["rows"]).to(torch.bfloat16)
        for b, (path, _) in enumerate(walked):
            n = int(s.context[b])
            at = int(starts[b])
            for pool in range(2 * LAYERS):
                now = rows_at(s, pool, b, n)
                before = have[b][pool]
                assert torch.equal(now[: len(before)], before.to(now.dtype))
                if len(path):
                    fresh = wide[pool // 2, at:at + new[b]][path]
                    fresh = fresh[:, HEADS * RATIO + HEADS:] if pool % 2 else fresh[:, HEADS * RATIO:HEADS * RATIO + HEADS]
                    got = now[len(before):].view(s.pools[0].dtype).to(torch.float64).numpy()
                    if pool % 2:
                        y, size = S.f64(fresh), np.abs(S.f64(fresh))
                    else:
                        y, size = S.norm_rotate(S.f64(fresh), S.f64(s.norms[1, pool // 2]), 1e-6, context[b] + np.arange(len(path)),
                                                S.f64(s.freq), False)
                    if kind == torch.bfloat16:
                        assert (np.abs(got - y) <= S.tolerance_bf16(y, size)).all()
                    else:
                        c = (s.scale["k_scale"], s.scale["v_scale"])[pool % 2]
                        assert (np.abs(got - np.clip(y / c, -448, 448)) <= S.tolerance_e4m3(y / c, size / c)).all()
                have[b][pool] = now
        # the pages that a request holds are those that its tokens need
        assert s.held.tolist() == [-(-int(c) // PAGE) for c in s.context.tolist()]
    assert int(s.count) == PAGES and sorted(s.free.tolist()) == list(range(PAGES)) and not s.extra.any()


def test_attention_of_a_forked_request(kvc, cuda):
    """The child's attention over shared and copied pages is its parent's."""
    s = Server(kvc, cuda, torch.bfloat16)
    rng = np.random.default_rng(8)
    for turn in range(3):
        context = s.context.cpu().numpy()
        _, host = step_inputs([12, 9, 0, 0, 0], context, rng)
        host["accept"][:] = 0                    # all of the first branch is kept
        for name, t in s.inputs.items():
            t.copy_(torch.from_numpy(host[name]))
        s.step()
        s.results()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)
    s.shared.fork(i32([0, 1, 0]), i32([2, 3, 4]), s.context)
    s.shared.result()
    s.context[2:] = s.context[[0, 1, 0]]
    q = torch.randn((2, HEADS * RATIO, D), device=cuda).to(torch.bfloat16)[[0, 1, 0, 1, 0]].contiguous()
    rows = torch.randn((2, HEADS, D), device=cuda).to(torch.bfloat16)[[0, 1, 0, 1, 0]].contiguous()
    s.tab(s.context, i32([1] * 5))
    assert s.tab.result() == 5
    kvc.kvc_paged_append(s.paged, 0, rows, rows, s.slots[:5])
    out, lse = s.att(0, q, s.starts, s.context)
    s.att.result()
    assert torch.equal(out[2:], out[[0, 1, 0]]) and torch.equal(lse[2:], lse[[0, 1, 0]])
    want = R.attention(R.to_f64(s.pools[0]), R.to_f64(s.pools[1]), s.table.cpu().numpy(), PAGE, R.to_f64(q), np.arange(6),
                       s.context.cpu().numpy(), np.ones((5, 1), np.uint64), D ** -0.5, 1.0)
    tol_out, tol_lse = R.tolerances(want[0], want[2], want[3], 100, D)
    assert (np.abs(R.to_f64(out) - want[0]) <= tol_out).all() and (np.abs(R.to_f64(lse) - want[1]) <= tol_lse).all()

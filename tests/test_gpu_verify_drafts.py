"""Verification of drafted tokens against the plain walk: every kept node and
every token equal; and that what comes out follows the target's distribution."""
import sys

import numpy as np
import pytest
import torch

import step_reference as S

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def tree_parents(n, rng, wide):
    """Parents of a tree's nodes: among the last `wide` nodes."""
    return np.array([-1] + [int(rng.integers(max(0, i - wide), i)) for i in range(1, n)])[:n]


class Case:
    """Inputs on the host; target and draft rows in wider rows that begin at
    any value."""

    def __init__(self, nodes, vocab, draft, wide, seed, pad=0, sharp=1.5, more_rows=0):
        rng = np.random.default_rng(seed)
        self.nodes, self.vocab = np.array(nodes), vocab
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        rows = self.rows = int(self.starts[-1]) + more_rows
        x = rng.standard_normal((rows, vocab)) * sharp
        self.target = self.softmax(x)
        self.draft = self.softmax(x + 0.5 * rng.standard_normal((rows, vocab))) if draft else None
        self.parents = None if wide == 0 else np.concatenate([tree_parents(n, rng, wide) for n in nodes] +
                                                             [np.full(more_rows, 77)]).astype(np.int32)
        self.tokens = np.full(rows, 12345678, np.int32)          # (a first node's is not looked at)
        for b, n in enumerate(nodes):
            for i in range(1, n):
                up = self.starts[b] + (i - 1 if self.parents is None else self.parents[self.starts[b] + i])
                law = (self.draft if draft else self.target)[up].astype(np.float64)
                self.tokens[self.starts[b] + i] = rng.choice(vocab, p=law / law.sum())
        self.accept = rng.random(rows, dtype=np.float32)
        self.sample = rng.random(len(nodes), dtype=np.float32)
        self.pad = pad

    @staticmethod
    def softmax(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    def wide_rows(self, x, cuda):
        if x is None:
            return None
        rows, stride = x.shape[0], self.vocab + self.pad
        flat = torch.full((rows * stride + self.pad,), float("nan"), device=cuda)
        view = flat[self.pad:].view(rows, stride)[:, :self.vocab]
        view.copy_(torch.from_numpy(x))
        return view

    def args(self, cuda):
        d = lambda x: None if x is None else torch.from_numpy(x).to(cuda)
        return dict(target=self.wide_rows(self.target, cuda), tokens=d(self.tokens), row_starts=d(self.starts),
                    accept=d(self.accept), sample=d(self.sample), parents=d(self.parents),
                    draft=self.wide_rows(self.draft, cuda))

    def want(self):
        kept, lens, out = np.full(self.rows, -1), [], np.full(self.rows, -1)
        for s, (path, tokens) in zip(self.starts, S.verify(self.starts, self.tokens, self.parents, self.target, self.draft,
                                                           self.accept, self.sample)):
            kept[s:s + len(path)], out[s:s + len(tokens)] = path, tokens
            lens.append(len(path))
        return kept, np.array(lens), out

    def check(self, got, sequences=None):
        kept, lens, out = (t.cpu().numpy() for t in got)
        want = self.want()
        which = range(len(self.nodes)) if sequences is None else sequences
        for b in which:
            s, e = self.starts[b], self.starts[b + 1]
            assert lens[b] == want[1][b], b
            assert np.array_equal(kept[s:e], want[0][s:e]), b
            assert np.array_equal(out[s:e], want[2][s:e]), b

    def run(self, kvc, cuda, verifier=None, **kw):
        v = verifier or kvc.DraftVerifier(len(self.nodes), self.vocab, self.rows)
        got = v(**self.args(cuda), **kw)
        v.result()
        self.check(got)
        return got


@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 1000, 4095, 4096, 4097, 12289])
@pytest.mark.parametrize("draft,wide", [(True, 0), (False, 0), (False, 3), (True, 3)])
@pytest.mark.parametrize("pad", [0, 3])
def test_vocabularies_and_strides(kvc, cuda, vocab, draft, wide, pad):
    say(f"vocab {vocab} draft {draft} wide {wide} pad {pad}")
    Case([5, 1, 0, 9, 2], vocab, draft, wide, vocab + pad, pad).run(kvc, cuda)


@pytest.mark.parametrize("draft,wide", [(True, 0), (False, 0), (False, 4), (True, 4), (True, 1000), (False, 1000)])
@pytest.mark.parametrize("seed", range(4))
def test_batches(kvc, cuda, draft, wide, seed):
    """Many ragged sequences, chains, narrow trees and stars."""
    rng = np.random.default_rng(seed)
    nodes = rng.integers(0, 20, 60)
    Case(nodes, int(rng.integers(20, 700)), draft, wide, 100 + seed, sharp=2.5).run(kvc, cuda)


@pytest.mark.parametrize("draft,wide", [(True, 0), (False, 0), (False, 200), (True, 200), (False, 5)])
def test_long_sequences(kvc, cuda, draft, wide):
    """Up to the most nodes that a sequence may have, many children of one
    node, the same token drawn again and again."""
    Case([300, 1024, 65, 64], 30, draft, wide, 7, sharp=1.0).run(kvc, cuda)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("u", [0.0, 0.99999994, float("nan"), -1.0, 2.0])
def test_random_numbers_at_their_ends(kvc, cuda, draft, u):
    c = Case([8, 4], 5000, draft, 2, 9)
    c.accept[:] = np.float32(u)
    c.run(kvc, cuda)
    c = Case([8, 4], 5000, draft, 2, 9)
    c.sample[:] = np.float32(u)
    c.run(kvc, cuda)


def test_what_is_no_probability(kvc, cuda):
    """NaN and what is negative count as 0, what is over 1 as 1; where nothing
    is left the target's own row is drawn from."""
    for draft in (True, False):
        c = Case([6, 6, 6, 6, 6], 300, draft, 2, 10)
        c.target[0, 5:40], c.target[1, ::3], c.target[6, 7] = np.nan, -0.5, np.inf
        c.target[12:18] = 0
        c.target[12:18, 17] = 1                  # all that is left after a rejection of 17 is nothing
        c.tokens[13:18] = 17
        c.accept[13:18] = 2.0
        if draft:
            c.draft[12:18] = c.target[12:18]
            c.draft[18:24] = c.target[18:24]
            c.accept[18:24] = 1.5
            c.draft[1, 10:20], c.draft[2, 30] = np.nan, np.inf
        c.run(kvc, cuda)


def test_a_row_without_probabilities(kvc, cuda):
    c = Case([1, 3, 2], 100, False, 0, 11)
    c.target[0] = 0
    v = kvc.DraftVerifier(3, 100, 6)
    got = v(**c.args(cuda))
    with pytest.raises(kvc.KvcError) as e:
        v.result()
    assert e.value.status == kvc.KVC_ERR_INVALID
    c.check(got)
    assert got[2][0] == -1
    c.target[0, 3] = 1
    c.run(kvc, cuda, v)


def test_what_does_not_fit(kvc, cuda):
    """The bad sequence is reported, the others are right; rows behind the
    last one are left as they were."""
    def refused(c, bad, touched=True):
        v = kvc.DraftVerifier(len(c.nodes), c.vocab, c.rows)
        outs = [torch.full((n,), -9, dtype=torch.int32, device=cuda) for n in (c.rows, len(c.nodes), c.rows)]
        got = v(**c.args(cuda), kept=outs[0], kept_lens=outs[1], out_tokens=outs[2])
        with pytest.raises(kvc.KvcError) as e:
            v.result()
        assert e.value.status == kvc.KVC_ERR_INVALID
        c.check(got, [b for b in range(len(c.nodes)) if b not in bad])
        return got

    for draft in (True, False):
        c = Case([4, 4, 4], 50, draft, 2, 12)
        c.parents[5], c.parents[6] = 1, 3        # not before its node
        refused(c, [])
        c = Case([4, 4, 4], 50, draft, 2, 12)
        c.parents[9] = -3
        refused(c, [])
        c = Case([4, 4, 4], 50, draft, 2, 13)
        c.tokens[5], c.tokens[9], c.tokens[10] = 50, -1, 0x7FFFFFFF
        refused(c, [])
    c = Case([4, 4, 4], 50, True, 0, 14)
    c.starts = np.array([0, 4, 3, 12], np.int32)
    got = refused(c, [0, 1, 2])
    assert got[1].tolist()[1] == 0
    c = Case([4, 4, 4], 50, True, 0, 14)
    c.starts = np.array([0, 4, 8, 13], np.int32)
    got = refused(c, [2])
    assert got[1][2] == 0 and (got[0][8:] == -9).all() and (got[2][8:] == -9).all()
    c = Case([4, 4, 4], 50, True, 0, 14)
    c.starts = np.array([-1, 4, 8, 12], np.int32)
    refused(c, [0])
    c = Case([2, 1025], 9, False, 0, 15)
    got = refused(c, [1])
    assert got[1][1] == 0 and (got[0][2:] == -9).all()


def test_rows_behind_the_last(kvc, cuda):
    for draft in (True, False):
        c = Case([3, 0, 5], 200, draft, 2, 16, more_rows=4)
        outs = [torch.full((n,), -9, dtype=torch.int32, device=cuda) for n in (12, 3, 12)]
        c.run(kvc, cuda, kept=outs[0], kept_lens=outs[1], out_tokens=outs[2])
        assert (outs[0][8:] == -9).all() and (outs[2][8:] == -9).all()
    c = Case([0, 0], 200, True, 0, 17)
    assert c.run(kvc, cuda)[1].tolist() == [0, 0]


@pytest.mark.parametrize("mode", ["chain", "picked", "drawn"])
def test_tokens_follow_the_target(kvc, cuda, mode):
    """40000 sequences of one small tree: the first new token has the target's
    law behind node 0, and where a given one was kept the second has the law
    behind it; each count within 5 standard deviations (and one count)."""
    n, vocab, nodes = 40000, 6, 4
    rng = np.random.default_rng(5)
    p, q = rng.dirichlet(np.ones(vocab), nodes), rng.dirichlet(np.ones(vocab), nodes)
    parents = None if mode == "chain" else np.array([-1, 0, 0, 0])
    tokens = np.zeros((n, nodes), np.int32)
    for i in range(1, nodes):
        up = i - 1 if parents is None else 0
        tokens[:, i] = [2, 0, 2, 4][i] if mode == "picked" else rng.choice(vocab, n, p=q[up])
    # behind a kept node the law of that node's place is used, whatever its token
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda)
    target = dev(np.tile(p.astype(np.float32), (n, 1)))
    draft = None if mode == "picked" else dev(np.tile(q.astype(np.float32), (n, 1)))
    v = kvc.DraftVerifier(n, vocab, n * nodes)
    kept, lens, out = v(target, dev(tokens.reshape(-1)), dev(np.arange(n + 1, dtype=np.int32) * nodes),
                        dev(rng.random(n * nodes, dtype=np.float32)), dev(rng.random(n, dtype=np.float32)),
                        parents=None if parents is None else dev(np.tile(parents.astype(np.int32), n)), draft=draft)
    v.result()
    kept, lens, out = kept.view(n, nodes).cpu().numpy(), lens.cpu().numpy(), out.view(n, nodes).cpu().numpy()

    def follows(values, law):
        count = np.bincount(values, minlength=vocab)
        spread = np.sqrt(len(values) * law * (1 - law))
        assert (np.abs(count - len(values) * law) <= 5 * spread + 1).all(), (count, len(values) * law)

    follows(out[:, 0], p[0])
    assert (lens > 1).any() and (lens == 1).any()
    for node in range(1, nodes):
        second = out[(lens > 1) & (kept[:, 1] == node), 1]
        if len(second) > 100:
            follows(second, p[node])


@pytest.mark.parametrize("vocab", [65536, 61441, 100003])
@pytest.mark.parametrize("wide,noise", [(3, 0.5), (1000, 0.5), (4, 3.0)])
def test_drawn_trees_over_wide_vocabularies(kvc, cuda, vocab, wide, noise):
    """First rejections summed ahead: of deep trees, of stars with more
    children than are summed ahead for, of drafts that are rejected often, of
    more nodes than are looked at."""
    c = Case([9, 1, 0, 24, 70], vocab, True, wide, vocab + wide, pad=1, sharp=noise + 1)
    rng = np.random.default_rng(1)
    c.accept[:] = rng.random(len(c.accept), dtype=np.float32) ** np.float32(1 / noise)
    c.run(kvc, cuda)


def test_results_do_not_change_from_call_to_call(kvc, cuda):
    c = Case([9] * 40, 9000, True, 3, 18)
    v = kvc.DraftVerifier(40, 9000, 360)
    first = [t.clone() for t in c.run(kvc, cuda, v)]
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, c.run(kvc, cuda, v)))


@pytest.mark.parametrize("draft,wide", [(True, 0), (True, 3), (False, 3)])
def test_streams_and_graphs(kvc, cuda, draft, wide):
    """Two objects on two streams at once; two graphs of one object each,
    replayed in turn on new inputs."""
    cases = [Case([7, 3, 0, 12], 5000, draft, wide, 20 + i) for i in range(4)]
    objects = [kvc.DraftVerifier(4, 5000, 22) for _ in range(2)]
    args = [c.args(cuda) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [o(**a, stream=s) for o, a, s in zip(objects, args, streams)]
    for o, s, c, g in zip(objects, streams, cases, got):
        o.result(s)
        c.check(g)
    graphs, outs = [], []
    for o, a in zip(objects, args):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(o(**a))
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1):
            c = cases[(turn + i) % 4]
            for name, x in c.args(cuda).items():
                if x is not None:
                    args[i][name].copy_(x)
            graphs[i].replay()
            objects[i].result()
            c.check(outs[i])


def test_an_object_takes_fewer_rows(kvc, cuda):
    v = kvc.DraftVerifier(3, 700, 60)
    for nodes in ([20, 20, 20], [1, 1, 1], [0, 5, 2]):
        Case(nodes, 700, True, 2, sum(nodes)).run(kvc, cuda, v)


def test_refusals(kvc, cuda):
    c = Case([3, 2], 100, True, 2, 30)
    ok = c.args(cuda)
    v = kvc.DraftVerifier(2, 100, 5)
    for name, x in (("tokens", ok["tokens"].long()), ("row_starts", ok["row_starts"][:2]), ("accept", ok["accept"].double()),
                    ("sample", ok["sample"][:1]), ("parents", ok["parents"][:4]), ("target", ok["target"].bfloat16()),
                    ("target", ok["target"][:, :99]), ("target", ok["target"].t().contiguous().t()), ("draft", ok["draft"][:4]),
                    ("draft", ok["draft"].cpu()), ("kept", ok["tokens"][:3]), ("kept_lens", ok["tokens"]),
                    ("out_tokens", ok["tokens"].float())):
        with pytest.raises(ValueError):
            v(**{**ok, name: x})
    with pytest.raises(ValueError):
        kvc.DraftVerifier(2, 100, 4)(**ok)
    with pytest.raises(kvc.KvcError):
        v(**{**ok, "target": ok["target"][:1].expand(5, 100)})
    for bad in ((0, 100, 5), (2, 0, 5), (2, (1 << 20) + 1, 5), (2, 100, -1)):
        with pytest.raises(kvc.KvcError):
            kvc.DraftVerifier(*bad)


def test_the_widest_vocabulary(kvc, cuda):
    """2^20 tokens, all of them likely beyond measure: sums near 2^62."""
    vocab = 1 << 20
    for draft in (False, True):
        c = Case([3], 4, draft, 2, 31)
        c.vocab = vocab
        rng = np.random.default_rng(1)
        c.target = np.ones((3, vocab), np.float32)
        c.target[0] = rng.random(vocab, dtype=np.float32)
        c.draft = np.full((3, vocab), 0.25, np.float32) if draft else None
        c.parents[1:] = 0
        c.tokens[1:] = [5, vocab - 1]
        c.accept[1:] = [4.5, 9.0]
        c.run(kvc, cuda)

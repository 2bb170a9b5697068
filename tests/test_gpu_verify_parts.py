"""Verification where a sequence's vocabulary is split over few workgroups, so
that each of them sums several chunks and the last one fewer: drawn trees with
and without their first rejections summed ahead, second rejections beside them,
more than 64 chunks, batches larger than a launch has workgroups; and row
starts that do not begin with row 0."""
import numpy as np
import pytest
import torch

import step_reference as S
from test_gpu_paged_share import Cache, dev
from test_gpu_verify_drafts import Case

pytestmark = pytest.mark.gpu

CHUNK = 4096


def parts_of(groups, batch, vocab):
    """(workgroups of a sequence, chunks of each, of the last one), as the launch has them."""
    chunks = -(-vocab // CHUNK)
    parts = min(max(groups // batch, -(-chunks // 64)), chunks)
    per = -(-chunks // parts)
    parts = -(-chunks // per)
    return parts, per, chunks - per * (parts - 1)


@pytest.mark.parametrize("nodes,vocab,ahead,drawn", [
    ([3] * 70, 66001, (9, 2, 1), (3, 6, 5)),         # first rejections ahead; parts of several chunks, the last shorter
    ([3, 2, 4, 1, 0] * 30, 61441, (6, 3, 1), (1, 16, 16)),
    ([3] * 21, 397313, (33, 3, 2), (11, 9, 8)),
    ([2] * 135, 266241, (7, 10, 6), (2, 33, 33)),   # two workgroups at least: a workgroup sums at most 64 chunks
    ([6, 2, 5] * 13, 60000, None, (1, 15, 15)),      # none ahead; the only workgroup's turns of four chunks
    ([4, 7] * 10, 58000, None, (3, 5, 5)),
])
def test_drawn_trees_of_several_chunks_a_part(kvc, cuda, nodes, vocab, ahead, drawn):
    batch, wide = len(nodes), -(-vocab // CHUNK) >= 16
    assert wide == (ahead is not None)
    if wide:
        assert parts_of(1024, batch, vocab) == ahead
    assert parts_of(256 if wide else 64, batch, vocab) == drawn
    c = Wide(nodes, vocab, batch + vocab)
    walked = S.verify(c.starts, c.tokens, c.parents, c.target, c.draft, c.accept, c.sample)
    v = kvc.DraftVerifier(batch, vocab, c.rows)
    got = v(**c.args(cuda))
    v.result()
    kept, lens, out = (t.cpu().numpy() for t in got)
    for b, (path, tokens) in enumerate(walked):
        at, n = int(c.starts[b]), int(nodes[b])
        assert lens[b] == len(path), b
        assert kept[at:at + n].tolist() == path + [-1] * (n - len(path)), b
        assert out[at:at + n].tolist() == tokens + [-1] * (n - len(tokens)), b


class Wide(Case):
    """Trees in which every node hangs on node 0 or 1, rejected about every
    other time; probabilities float32 throughout (wide rows would take
    gigabytes in float64)."""

    def __init__(self, nodes, vocab, seed):
        rng = np.random.default_rng(seed)
        self.nodes, self.vocab, self.pad = np.array(nodes), vocab, 1
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        rows = self.rows = int(self.starts[-1])
        self.target = rng.random((rows, vocab), dtype=np.float32) ** 4
        self.draft = self.target + rng.random((rows, vocab), dtype=np.float32) ** 4
        for x in (self.target, self.draft):
            x /= x.sum(-1, keepdims=True)
        self.parents = np.concatenate([[-1] + [int(rng.integers(0, min(i, 2))) for i in range(1, n)]
                                       for n in nodes if n]).astype(np.int32)
        self.tokens = np.zeros(rows, np.int32)
        for b, n in enumerate(nodes):
            for i in range(1, n):
                law = np.cumsum(self.draft[self.starts[b] + self.parents[self.starts[b] + i]], dtype=np.float64)
                self.tokens[self.starts[b] + i] = min(int(np.searchsorted(law, rng.random() * law[-1], "right")), vocab - 1)
        self.accept = np.sqrt(rng.random(rows, dtype=np.float32))
        self.sample = rng.random(len(nodes), dtype=np.float32)


@pytest.mark.parametrize("siblings", [2, 3, 6, 12])
def test_rejections_of_siblings_ahead_and_behind(kvc, cuda, siblings):
    """Stars whose children are all rejected: the first rejection summed ahead,
    the others by the walk, and both give one distribution."""
    c = Wide([siblings + 1] * 9, 65537 + siblings, siblings)
    c.parents[:] = np.tile([-1] + [0] * siblings, 9)
    c.accept[:] = np.float32(0.99999994)
    for b in range(9):                           # tokens that the draft has more often than the target
        more = np.argsort(c.draft[c.starts[b]] - c.target[c.starts[b]])[-4 * siblings:]
        c.tokens[c.starts[b] + 1:c.starts[b + 1]] = more[::4]
    walked = S.verify(c.starts, c.tokens, c.parents, c.target, c.draft, c.accept, c.sample)
    assert sum(len(path) == 1 for path, _ in walked) >= 3
    c.run(kvc, cuda)


@pytest.mark.parametrize("batch,vocab,parts", [(1100, 1 << 18, (1, 64, 64)), (600, 70001, (1, 18, 18)), (400, 70001, (2, 9, 9))])
def test_batches_past_a_launch(kvc, cuda, batch, vocab, parts):
    """One node a sequence: the draw alone, of workgroups that sum up to 64
    chunks."""
    assert parts_of(1024, batch, vocab) == parts
    rng = np.random.default_rng(batch)
    law = rng.random((7, vocab), dtype=np.float32) ** 8
    law /= law.sum(-1, keepdims=True)
    target = torch.from_numpy(law).to(cuda)[torch.arange(batch, device=cuda) % 7]
    sample = rng.random(batch, dtype=np.float32)
    v = kvc.DraftVerifier(batch, vocab, batch)
    kept, lens, out = v(target, torch.zeros(batch, dtype=torch.int32, device=cuda),
                        torch.arange(batch + 1, dtype=torch.int32, device=cuda), torch.zeros(batch, device=cuda), dev(sample, cuda))
    v.result()
    upto = np.cumsum(S.units(law), -1)
    point = (sample.astype(np.float64) * upto[np.arange(batch) % 7, -1]).astype(np.int64)
    want = [int(np.searchsorted(upto[b % 7], min(point[b], upto[b % 7, -1] - 1), "right")) for b in range(batch)]
    assert (kept == 0).all() and (lens == 1).all() and out.tolist() == want


@pytest.mark.parametrize("draft,wide", [(True, 0), (True, 3), (False, 3)])
def test_rows_in_front_of_the_first(kvc, cuda, draft, wide):
    c = Case([2, 5, 3, 8], 3000, draft, wide, 41)
    c.starts, c.nodes, c.sample = c.starts[1:], c.nodes[1:], c.sample[1:]
    outs = [torch.full((n,), -9, dtype=torch.int32, device=cuda) for n in (c.rows, 3, c.rows)]
    c.run(kvc, cuda, kept=outs[0], kept_lens=outs[1], out_tokens=outs[2])
    assert (outs[0][:2] == -9).all() and (outs[2][:2] == -9).all()


def test_compaction_of_rows_in_front_of_the_first(kvc, cuda):
    c = Cache(kvc, cuda, [2, 3], 8, 2, 2, 64, "bf16", 42)
    starts, context, lens = np.array([4, 11, 20], np.int32), np.array([9, 15], np.int32), np.array([3, 4], np.int32)
    kept = np.full(22, 77, np.int32)
    kept[4:7], kept[11:15] = [0, 2, 6], [1, 2, 5, 8]
    op = kvc.PagedCompaction(c.paged)
    op(*(dev(x, cuda) for x in (starts, context, kept, lens)))
    op.result()
    S.compact(c.pools.numpy(), c.table, 8, starts, context, kept, lens)
    c.same_pools()

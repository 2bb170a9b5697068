"""Infinities and NaN in V of the tokens that a row sees: in the context
beside drafted ones, and in tokens of hardly any weight."""
import sys

import numpy as np
import pytest
import torch

import paged_reference as R
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def plant(c, b, pos, x, head=slice(None), ch=slice(None)):
    """V of token `pos` of sequence b becomes x (NaN for an infinity of e4m3,
    which has none)."""
    v = c.pools[2 * c.layer + 1]
    if v.dtype != torch.bfloat16:
        x = NAN
    v[int(c.table[b, pos // c.page]), pos % c.page, head, ch] = x


def check(c, got, clean):
    """Against float64 on the same values: what is not finite there is the
    same here, and the rest is within the tolerances of the values without
    them."""
    with np.errstate(invalid="ignore"):
        out, lse = c.ref()[:2]
    special = ~np.isfinite(out)
    assert special.any() and not special.all()
    tol_out, tol_lse = R.tolerances(np.where(special, 0.0, out), clean[2], clean[3],
                                    int((c.contexts + c.nodes).max()), c.d)
    o, z = R.to_f64(got[0]), R.to_f64(got[1])
    assert np.array_equal(np.isnan(o), np.isnan(out)), np.argwhere(np.isnan(o) != np.isnan(out))[:4]
    assert np.array_equal(o[np.isinf(out)], out[np.isinf(out)])
    assert (np.abs(o[~special] - out[~special]) <= tol_out[~special]).all()
    seen = ~np.isneginf(lse)
    assert (np.abs(z[seen] - lse[seen]) <= tol_lse[seen]).all()


@pytest.mark.parametrize("hint", [1, 64])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 12, 7])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_context_values_beside_drafted_ones(kvc, cuda, d, page, kind, hint):
    """A tile of context and drafted tokens with such values in both: every
    row has those of the context, the rows that see the drafted token its
    own; in one workgroup and in a sequence that several share."""
    print(f"case {d} {page} {kind} {hint}", file=sys.stderr, flush=True)
    for tree in (True, False):
        c = Case(kvc, cuda, [20, 1300 + d, 45], [9, 6, 3], 2, 2, d, kind, page, tree, seed=41)
        clean = c.ref()
        for b, drafted in ((0, 1), (1, 3), (2, 2)):
            ctx = int(c.contexts[b])
            plant(c, b, ctx - 3, NAN, 0, 3)
            plant(c, b, ctx - 1, INF, 1, d - 1)
            plant(c, b, ctx + drafted, INF, slice(None), 9)
            plant(c, b, ctx + drafted, NAN, 0, 20)
        for most in (0, 60):
            check(c, c.run(hint=hint, most=most), clean)


@pytest.mark.parametrize("hint", [1, 64])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("nodes", [[3, 2], [100, 70]])
def test_drafted_values_of_hardly_any_weight(kvc, cuda, nodes, tree, kind, hint):
    """The drafted tokens' scores lie 400 below the first tokens': their
    weights are 0 in float32, in a tile of their own, in a part of the
    sequence of their own and in its join.  What is infinite in them is
    infinite in the rows that see it (and nothing else changes)."""
    c = Case(kvc, cuda, [2048, 33], nodes, 2, 2, 128, kind, 16, tree, seed=42, scale=1.0)
    one = torch.zeros(128, device=cuda)
    one[5] = 1.0
    k = c.pools[2 * c.layer]
    for b, high in ((0, 700), (1, 32)):
        for pos in range(int(c.contexts[b]) + nodes[b]):
            k[int(c.table[b, pos // 16]), pos % 16] = ((10.0 if pos < high else -10.0) * one).to(k.dtype)
    c.q = (20.0 * one + 0.01 * c.q.float()).to(torch.bfloat16)
    clean = c.ref()
    for b in range(2):
        ctx = int(c.contexts[b])
        plant(c, b, ctx, INF, 0, 9)
        plant(c, b, ctx + nodes[b] - 1, -INF, 1, 100)
        plant(c, b, ctx + nodes[b] // 2, NAN, 1, 64)
    for most in (0, 60):
        check(c, c.run(hint=hint, most=most), clean)

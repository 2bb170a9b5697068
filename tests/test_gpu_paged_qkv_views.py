"""Norms, rotation and append of rows that lie in every way that strides can
say: heads apart, rows and heads that are one, queries written into wider rows
and over themselves."""
import pytest
import torch

import test_gpu_paged_qkv

pytestmark = pytest.mark.gpu


class Case(test_gpu_paged_qkv.Case):
    def check(self, *args, **kw):
        self.v = self.v.contiguous()             # (the append, which the values are held to, takes whole rows)
        super().check(*args, **kw)


def heads_first(t):
    """The same values, each head's rows together."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("pool,d,heads,q_heads,interleaved", [
    ("bf16", 128, 4, 8, False), ("e4m3", 64, 8, 24, True), ("bf16", 192, 3, 7, True), ("e4m3", 256, 1, 5, False),
])
@pytest.mark.parametrize("rows", [1, 37, 1500])
def test_heads_apart(kvc, cuda, rows, pool, d, heads, q_heads, interleaved):
    c = Case(kvc, cuda, rows, q_heads, heads, d, 16, pool, d // 2, interleaved, "bf16", False, rows + d)
    c.q, c.k, c.v = heads_first(c.q), heads_first(c.k), heads_first(c.v)
    c.run()


def test_rows_and_heads_that_are_one(kvc, cuda):
    """Broadcast rows and heads: strides of 0."""
    c = Case(kvc, cuda, 50, 8, 4, 128, 16, "bf16", 128, False, "bf16", False, 1)
    c.q, c.k, c.v = c.q[:1].expand(50, -1, -1), c.k[:, :1].expand(-1, 4, -1), c.v[:1, :1].expand(50, 4, -1)
    keep = [p.clone() for p in c.pools]
    out = torch.full((50, 8, 128), 3.0, dtype=torch.bfloat16, device=cuda)
    before = out.clone()
    c.op()(1, c.q, c.k, c.v, c.slots.to(cuda), c.positions.to(cuda), out=out)
    c.check(1, out, before, keep)


@pytest.mark.parametrize("q_heads,heads", [(8, 2), (5, 3)])
@pytest.mark.parametrize("rows", [3, 900])
def test_queries_into_wider_rows(kvc, cuda, rows, q_heads, heads):
    """... and what lies beside them stays."""
    c = Case(kvc, cuda, rows, q_heads, heads, 64, 16, "bf16", 64, False, "f32", True, 2)
    wide = torch.full((rows, q_heads + 3, 64), 7.0, dtype=torch.bfloat16, device=cuda)
    out, keep = wide[:, 2:2 + q_heads], [p.clone() for p in c.pools]
    c.op()(0, c.q, c.k, c.v, c.slots.to(cuda), c.positions.to(cuda), out=out)
    c.check(0, out, torch.full_like(out, 7.0), keep)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + q_heads:] == 7).all()


@pytest.mark.parametrize("rows,q_heads,d", [(1, 8, 128), (700, 7, 192), (3000, 24, 64)])
def test_queries_over_themselves(kvc, cuda, rows, q_heads, d):
    """A projection's rows in place, whole rows to a wave and in parts."""
    c = Case(kvc, cuda, rows, q_heads, 2, d, 16, "e4m3", d, True, "bf16", True, 3)
    keep, before = [p.clone() for p in c.pools], c.q.clone()
    k, v = c.k.clone(), c.v.clone()
    c.op()(1, c.q, c.k, c.v, c.slots.to(cuda), c.positions.to(cuda), out=c.q)
    c.check(1, c.q, before, keep, q=before)
    assert torch.equal(c.k, k) and torch.equal(c.v, v)


def test_a_layers_own_norms(kvc, cuda):
    """Every layer's weights are its own, in the last layer too."""
    c = Case(kvc, cuda, 20, 4, 2, 128, 16, "bf16", 128, False, "f32", False, 4, layers=5)
    for layer in (0, 4, 2):
        c.run(layer)

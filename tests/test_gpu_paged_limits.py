"""Calls at the edge of what the paged cache's operators take."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_items_than_a_launch_has_workgroups_for(kvc, cuda):
    """1024 sequences of 16384 KV heads, one token each: a row sees that token
    alone, and its output is the token's V, bit for bit."""
    batch, heads, d = 1024, 16384, 64
    g = torch.Generator(device=cuda).manual_seed(61)
    v = torch.randn((batch, 1, heads, d), generator=g, device=cuda, dtype=torch.bfloat16)
    table = torch.randperm(batch, generator=g, device=cuda).to(torch.int32)[:, None]
    q = torch.randn((batch, heads, d), generator=g, device=cuda, dtype=torch.bfloat16)
    paged = kvc.PagedKV([q.view(batch, 1, heads, d), v], table, 1)
    starts = torch.arange(batch + 1, dtype=torch.int32, device=cuda)
    out, lse = kvc.kvc_paged_attention(paged, 0, q, starts)
    assert torch.equal(out, v[table[:, 0].long(), 0])
    k = paged.pools[0][table[:, 0].long(), 0].float()
    # 64 products of up to 6 x 6 summed in float32, scaled
    assert ((q.float() * k).sum(-1) * d ** -0.5 - lse).abs().max() < 80 * 2.0 ** -24 * 64 * 36 / 8

"""The paged-cache operators that stand around kvc_decode_paged: block tables and slot maps built from request lengths,
new K/V rows appended to the pages, and attention of drafted tokens over the pages.

Each case is one call of a serving step on one layer, with the head shapes of this repository's workloads (8 KV heads of
128 channels, 2 to 8 query heads a KV head) and a few generic ones.  Lengths of a batch are drawn from the case's own
`lens` seed, so that a case is the same work whatever the seed of its values.
"""
import math

import numpy as np
import torch

own = False

FP8_MAX = 448.0


# ---------------------------------------------------------------- cases

def _table(name, batch, page, cached, new, trim, max_tokens, lens, pad=0):
    return {"name": name, "op": "table", "batch": batch, "page": page, "cached": cached, "new": new, "trim": trim,
            "max_tokens": max_tokens, "lens": lens, "pad": pad}


def _append(name, rows, heads, dim, src, pool, page, strided, skip, lens):
    return {"name": name, "op": "append", "rows": rows, "heads": heads, "dim": dim, "src": src, "pool": pool,
            "page": page, "strided": strided, "skip": skip, "lens": lens}


def _attend(name, batch, nodes, tree, context, ragged, heads, ratio, dim, pool, page, lens):
    return {"name": name, "op": "attend", "batch": batch, "nodes": nodes, "tree": tree, "context": context,
            "ragged": ragged, "heads": heads, "ratio": ratio, "dim": dim, "pool": pool, "page": page, "lens": lens}


def listed():
    return [
        # one decode step of a small batch: the next token's page and slot of 8 requests (latency)
        _table("table 8 x 1", 8, 16, 4096, 1, False, 8192, 1),
        # a speculative step of a full server: 256 requests with up to 64 drafted tokens, finished ones give pages back
        _table("table 256 trees", 256, 16, 8192, 64, True, 32768, 2, 500),
        # admission of 64 prompts of up to 32K tokens into an empty cache
        _table("table 64 prompts", 64, 16, 0, 32768, False, 32768, 3),
        # one decode step of 4 sequences on one layer (latency)
        _append("append 4 rows", 4, 8, 128, "bf16", "bf16", 16, False, 0.0, 4),
        # a prompt's K/V, views of a fused projection, kept as bf16 pages
        _append("append prompt", 16384, 8, 128, "bf16", "bf16", 16, True, 0.0, 5),
        # an odd number of rows of a padded step rounded to an e4m3 cache
        _append("append e4m3", 8191, 8, 128, "bf16", "e4m3", 16, True, 0.1, 6),
        # the next token of one short sequence (the smallest model's heads; latency)
        _attend("attend 1 x 1 x 512", 1, 1, False, 512, False, 8, 2, 128, "bf16", 16, 7),
        # the next tokens of the 4 x 4096 cache
        _attend("attend 4 x 1 x 4096", 4, 1, False, 4096, False, 8, 4, 128, "bf16", 16, 8),
        # 16 drafted tokens a sequence over the same cache
        _attend("attend 4 x 16 x 4096", 4, 16, True, 4096, False, 8, 4, 128, "bf16", 16, 9),
        # a wide tree over the 32K-token cache, 8 query heads a KV head
        _attend("attend 1 x 64 x 32768", 1, 64, True, 32768, False, 8, 8, 128, "bf16", 16, 10),
        # a ragged batch with trees over an e4m3 cache in pages of 24 tokens
        _attend("attend 48 ragged e4m3", 48, 24, True, 8192, True, 8, 4, 128, "e4m3", 24, 11),
        # a piece of a prompt attending to what is cached and to itself
        _attend("attend chunk 1000", 2, 1000, False, 7001, False, 8, 4, 128, "bf16", 16, 12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "append", "attend", "attend"])
    lens = rng.randrange(1 << 30)
    if op == "table":
        batch = _log_int(rng, 1, 512)
        page = rng.choice([8, 16, 16, 24, 32, 64, 100])
        prompt = rng.random() < 0.5
        new = _log_int(rng, 64, max(64, min(32768, (1 << 20) // batch))) if prompt else _log_int(rng, 1, 64)
        cached = 0 if prompt else _log_int(rng, 16, 16384)
        c = _table("", batch, page, cached, new, rng.random() < 0.5, 2 * (cached + new), lens, rng.randrange(100))
    elif op == "append":
        src, pool = rng.choice([("bf16", "bf16"), ("bf16", "e4m3"), ("e4m3", "e4m3")])
        c = _append("", _log_int(rng, 1, 16384), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 192, 256]), src, pool,
                    rng.choice([1, 8, 16, 24, 64]), rng.random() < 0.5, rng.choice([0.0, 0.2]), lens)
    else:
        batch = _log_int(rng, 1, 48)
        nodes = _log_int(rng, 1, max(1, min(128, 1024 // batch)))
        dim = rng.choice([64, 128, 128, 192, 256])
        heads = rng.choice([1, 2, 4, 8])
        c = _attend("", batch, nodes, nodes > 1 and rng.random() < 0.75, _log_int(rng, 8, min(32768, 131072 // batch)),
                    rng.random() < 0.5, heads, rng.choice([1, 2, 4, 5, 8]), dim, rng.choice(["bf16", "e4m3"]),
                    rng.choice([8, 16, 16, 24, 32, 64, 128]), lens)
    del c["name"]
    return c


def _lengths(case):
    """(cached or context, new or drafted) lengths of the batch, of the case alone."""
    r = np.random.RandomState(case["lens"] % (1 << 31))
    b = case["batch"]
    if case["op"] == "table":
        cached = r.randint(case["cached"] // 4, case["cached"] + 1, b)
        new = r.randint(max(1, case["new"] // 4), case["new"] + 1, b)
        if case["trim"]:                       # a tenth of the requests are finished, others lost what was rejected
            done = r.rand(b) < 0.1
            cached[done] = 0
            new[done] = 0
        return cached, new
    if case["ragged"]:
        return r.randint(0, case["context"] + 1, b), r.randint(1, case["nodes"] + 1, b)
    return np.full(b, case["context"]), np.full(b, case["nodes"])


def _held(case, cached):
    """Pages that each request holds before the call: those of its cached tokens, and with trim some more."""
    r = np.random.RandomState((case["lens"] + 1) % (1 << 31))
    held = -(-cached // case["page"])
    if case["trim"]:
        most = -(-case["max_tokens"] // case["page"])
        held = np.minimum(held + r.randint(0, 9, len(held)), most)
    return held


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _values(shape, kind, g):
    """K or V rows: normal with a scale for each channel (the workloads' law)."""
    s = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    x = torch.randn(shape, generator=g, device="cuda").mul_(s)
    return x.to(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def _prepare_table(case, g):
    cached, new = _lengths(case)
    held = _held(case, cached)
    page, batch = case["page"], case["batch"]
    max_pages = -(-case["max_tokens"] // page)
    num_pages = int(held.sum() + (-(-(cached + new) // page)).sum()) + 17
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(max_pages, device="cuda")[None, :]
    used = col < _ints(held)[:, None]
    table[used] = perm[: int(held.sum())]
    n_free = num_pages - int(held.sum())
    free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_free] = perm[int(held.sum()):]
    rows = int(new.sum()) + case["pad"]
    return {"table": table, "free": free, "count": _ints([n_free]), "held": _ints(held), "cached": _ints(cached),
            "new": _ints(new), "num_pages": num_pages, "rows": rows}


def _prepare_append(case, g):
    rows, h, d = case["rows"], case["heads"], case["dim"]
    num_pages = -(-rows // case["page"]) + 5
    pools = [_values((num_pages, case["page"], h, d), case["pool"], g) for _ in range(2)]
    if case["strided"]:                        # K and V as views of one projection's rows, with the queries before them
        wide = _values((rows, 4 * h, d), case["src"], g)
        k, v = wide[:, 2 * h:3 * h], wide[:, 3 * h:]
    else:
        k, v = _values((rows, h, d), case["src"], g), _values((rows, h, d), case["src"], g)
    slots = torch.randperm(num_pages * case["page"], generator=g, device="cuda")[:rows]
    slots = torch.where(torch.rand(rows, generator=g, device="cuda") < case["skip"], torch.full_like(slots, -1), slots)
    scale = (0.75, 0.4) if case["pool"] != case["src"] else (1.0, 1.0)
    return {"pools": pools, "k": k, "v": v, "slots": slots, "scale": scale}


def _tree_masks(nodes, words, g):
    """Visible drafted tokens of every row, as bits: a node sees itself and its ancestors; parents are drawn among the
    nodes before it.  [batch * longest] rows, later packed."""
    batch, n = len(nodes), int(max(nodes))
    parent = (torch.rand((batch, n), generator=g, device="cuda") * torch.arange(n, device="cuda")).long()
    see = torch.zeros((batch, n, words), dtype=torch.int64, device="cuda")
    for i in range(n):
        if i:
            see[:, i] = see.gather(1, parent[:, i, None, None].expand(batch, 1, words))[:, 0]
        see[:, i, i // 64] |= -(1 << 63) if i % 64 == 63 else 1 << (i % 64)
    keep = torch.arange(n, device="cuda")[None, :] < _ints(nodes)[:, None]
    return see[keep].contiguous()


def _prepare_attend(case, g):
    context, nodes = _lengths(case)
    page, h, d = case["page"], case["heads"], case["dim"]
    total = context + nodes
    pages = -(-total // page)
    max_pages = int(pages.max()) + 2
    num_pages = int(pages.sum()) + 3
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["batch"], max_pages), dtype=torch.int32, device="cuda")
    used = torch.arange(max_pages, device="cuda")[None, :] < _ints(pages)[:, None]
    table[used] = perm[: int(pages.sum())]
    pools = [_values((num_pages, page, h, d), case["pool"], g) for _ in range(2)]
    rows = int(nodes.sum())
    q = torch.randn((rows, h * case["ratio"], d), generator=g, device="cuda").to(torch.bfloat16)
    words = -(-case["nodes"] // 64)
    return {"pools": pools, "tab": table, "q": q, "context": _ints(context), "nodes": _ints(nodes),
            "starts": _ints(np.concatenate([[0], np.cumsum(nodes)])),
            "mask": _tree_masks(nodes, words, g) if case["tree"] else None, "most": int(nodes.max()),
            "longest": int(total.max())}


def prepare(case, seed):
    g = _gen(seed)
    s = {"table": _prepare_table, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, g)
    s["case"] = case
    if case["op"] == "table":
        s["held_out"], s["count_out"] = torch.empty_like(s["held"]), torch.empty_like(s["count"])
        s["row_starts"] = torch.empty(case["batch"] + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(s["rows"], dtype=torch.int64, device="cuda")
        s["positions"] = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
    if own:                                    # the handles that a serving program keeps
        from entropy_coding_amd import kvc
        if case["op"] == "table":
            s["op"] = kvc.BlockTable(s["table"], s["held"], s["free"], s["count"], case["page"], s["num_pages"],
                                     s["row_starts"], s["slots"], s["positions"], held_out=s["held_out"],
                                     free_count_out=s["count_out"])
        elif case["op"] == "append":
            any_table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
            s["paged"] = kvc.PagedKV(s["pools"], any_table, case["page"])
        else:
            s["paged"] = kvc.PagedKV(s["pools"], s["tab"], case["page"])
            s["op"] = kvc.PagedAttention(s["paged"], case["heads"] * case["ratio"], s["q"].shape[0],
                                         rows_per_sequence=s["most"], max_tokens=s["longest"])
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_table(s, case):
    page, table, free = case["page"], s["table"], s["free"]
    cached, new, held = s["cached"].long(), s["new"].long(), s["held"].long()
    batch, max_pages = table.shape
    need = (cached + new + page - 1) // page
    grow = (need - held).clamp(min=0)
    extra = (held - need).clamp(min=0) if case["trim"] else torch.zeros_like(held)
    count, n_grow, n_extra = s["count"].long()[0], grow.sum(), extra.sum()
    col = torch.arange(max_pages, device="cuda")[None, :]
    back = table[(col >= need[:, None]) & (col < (need + extra)[:, None])].flip(0)      # pages given back, last first
    place = torch.arange(free.numel(), device="cuda")
    stack = torch.cat([free, free.new_zeros(back.numel())])
    at = torch.arange(back.numel(), device="cuda") + count
    stack[at] = back
    takes = (col >= held[:, None]) & (col < need[:, None])
    k = (torch.cumsum(grow, 0) - grow)[:, None] + col - held[:, None]
    table.copy_(torch.where(takes, stack[(count + n_extra - 1 - k).clamp(0, stack.numel() - 1)], table))
    left = count + n_extra - n_grow
    free.copy_(torch.where((place >= count) & (place < left), stack[: free.numel()], free))
    s["held_out"].copy_(need if case["trim"] else torch.maximum(held, need))
    s["count_out"].copy_(left[None])
    ends = torch.cumsum(new, 0)
    s["row_starts"].copy_(torch.cat([ends.new_zeros(1), ends]))
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(ends, r, right=True)
    real, b = b < batch, b.clamp(max=batch - 1)
    pos = cached[b] + r - (ends - new)[b]
    slot = table[b, torch.where(real, pos, 0) // page].long() * page + pos % page
    s["slots"].copy_(torch.where(real, slot, -1))
    s["positions"].copy_(torch.where(real, pos, -1))


def _plain_append(s, case):
    h, d = case["heads"], case["dim"]
    there = s["slots"] >= 0
    at = s["slots"][there]
    for pool, x, scale in zip(s["pools"], (s["k"], s["v"]), s["scale"]):
        x = x[there]
        if x.dtype != pool.dtype:
            x = (x.float() / scale).clamp(-FP8_MAX, FP8_MAX).to(pool.dtype)
        kind = torch.int16 if pool.element_size() == 2 else torch.uint8
        pool.view(kind).view(-1, h, d)[at] = x.view(kind)


def _rows_of(pool, slot):
    """fp32 rows of the slots: [..., heads, D]."""
    kind = torch.int16 if pool.element_size() == 2 else torch.uint8
    flat = pool.view(kind).view(-1, *pool.shape[2:])
    return flat[slot].view(pool.dtype).float()


def _plain_attend(s, case):
    h, ratio, d, page = case["heads"], case["ratio"], case["dim"], case["page"]
    batch, n, length = case["batch"], s["most"], s["longest"]
    context, nodes = s["context"].long(), s["nodes"].long()
    t = torch.arange(length, device="cuda")
    slot = s["tab"].long()[:, t // page] * page + t % page
    slot = torch.where(t[None, :] < (context + nodes)[:, None], slot, 0)
    i = torch.arange(n, device="cuda")
    real = i[None, :] < nodes[:, None]
    row = torch.where(real, s["starts"].long()[:-1, None] + i[None, :], 0)                 # [batch, n]
    j = t[None, :] - context[:, None]                                                      # [batch, length]
    if s["mask"] is None:
        see = j[:, None, :] <= i[None, :, None]
    else:
        jj = j.clamp(0, 64 * s["mask"].shape[1] - 1)
        word = s["mask"][row].gather(2, (jj // 64)[:, None, :].expand(batch, n, length))
        see = ((word >> (jj % 64)[:, None, :]) & 1).bool()
    see = (j < 0)[:, None, :] | (see & (j < nodes[:, None])[:, None, :])
    see = see[:, None, :, None, :]                                                         # [batch, 1, n, 1, length]
    q = s["q"].float()[row].view(batch, n, h, ratio, d).transpose(1, 2).reshape(batch, h, n * ratio, d)
    k = _rows_of(s["pools"][0], slot).transpose(1, 2).contiguous()                         # [batch, heads, length, d]
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(d)).view(batch, h, n, ratio, length)
    del k
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _rows_of(s["pools"][1], slot).transpose(1, 2).contiguous()
    o = torch.matmul(p.view(batch, h, n * ratio, length), v).view(batch, h, n, ratio, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0]
    o = o.transpose(1, 2).reshape(batch, n, h * ratio, d)[real]
    return o.to(torch.bfloat16), lse.transpose(1, 2).reshape(batch, n, h * ratio)[real]


def run(state):
    s, case = state, state["case"]
    if case["op"] == "table":
        if own:
            s["op"](s["cached"], s["new"], trim=case["trim"])
        else:
            _plain_table(s, case)
        return {k: s[k] for k in ("table", "free", "held_out", "count_out", "row_starts", "slots", "positions")}
    if case["op"] == "append":
        if own:
            from entropy_coding_amd import kvc
            kvc.kvc_paged_append(s["paged"], 0, s["k"], s["v"], s["slots"], k_scale=s["scale"][0], v_scale=s["scale"][1])
        else:
            _plain_append(s, case)
        return {"k": s["pools"][0], "v": s["pools"][1]}
    if own:
        out, lse = s["op"](0, s["q"], s["starts"], s["context"], s["mask"], out=s["out"], lse=s["lse"])
    else:
        out, lse = _plain_attend(s, case)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- work and the 64-bit values

def work(case):
    if case["op"] == "table":
        cached, new = _lengths(case)
        held = _held(case, cached)
        need = -(-(cached + new) // case["page"])
        rows = int(new.sum()) + case["pad"]
        taken = int(np.maximum(need - held, 0).sum())
        given = int(np.maximum(held - need, 0).sum()) if case["trim"] else 0
        # lengths and held pages in, held pages and starts out; a page number read and written for each taken or given
        # back, one read for each page whose tokens are new; 8 bytes a slot and 4 a position
        return {"bytes": 20 * case["batch"] + 8 * (taken + given) + 12 * rows, "flops": 0}
    if case["op"] == "append":
        size = {"bf16": 2, "e4m3": 1}
        n = case["rows"] * (1.0 - case["skip"]) * case["heads"] * case["dim"] * 2
        return {"bytes": n * (size[case["src"]] + size[case["pool"]]) + 8 * case["rows"], "flops": 0}
    context, nodes = (x.astype(np.float64) for x in _lengths(case))
    h, qh, d = case["heads"], case["heads"] * case["ratio"], case["dim"]
    size = 2 if case["pool"] == "bf16" else 1
    tokens, rows = float((context + nodes).sum()), float(nodes.sum())
    # a tree's rows see their depth, about the logarithm of their place; a chain's rows see half of it
    drafted = nodes * np.log(nodes + 1.0) if case["tree"] else nodes * (nodes + 1.0) / 2
    pairs = float((nodes * context + drafted).sum())
    return {"bytes": 2 * tokens * h * d * size + 4 * tokens / case["page"] + rows * qh * (4 * d + 4),
            "flops": 4 * pairs * qh * d}


def exact(case, seed):
    if case["op"] == "table":
        return None                            # whole numbers: the plain form's have to be met
    g = _gen(seed)
    if case["op"] == "append":
        s = _prepare_append(case, g)
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        out = []
        for pool, x, scale in zip(s["pools"], (s["k"], s["v"]), s["scale"]):
            y = pool.double().reshape(-1, case["heads"], case["dim"])
            y[s["slots"][keep]] = (x[keep].double() / scale).clamp(-FP8_MAX, FP8_MAX)
            out.append(y.view(pool.shape))
        return {"k": out[0], "v": out[1]}
    s = _prepare_attend(case, g)
    context, nodes = _lengths(case)
    h, ratio, d, page = case["heads"], case["ratio"], case["dim"], case["page"]
    k_all, v_all = (p.view(-1, h, d) for p in s["pools"])
    outs, lses, r0 = [], [], 0
    for b in range(case["batch"]):
        c, n = int(context[b]), int(nodes[b])
        rows = torch.repeat_interleave(s["tab"][b, : -(-(c + n) // page)].long() * page, page)
        rows = (rows + torch.arange(page, device="cuda").repeat(rows.numel() // page))[: c + n]
        see = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        for i in range(n):
            if s["mask"] is None:
                see[i, c + i + 1:] = False
        if s["mask"] is not None:
            bits = s["mask"][r0:r0 + n][:, :, None] >> torch.arange(64, device="cuda")[None, None, :]
            see[:, c:] = (bits & 1).reshape(n, -1)[:, :n] == 1
        k, v = (x.view(torch.int16 if page and x.element_size() == 2 else torch.uint8)[rows].view(x.dtype).double()
                for x in (k_all, v_all))
        o = torch.empty((n, h * ratio, d), dtype=torch.float64, device="cuda")
        z = torch.empty((n, h * ratio), dtype=torch.float64, device="cuda")
        for a in range(h * ratio):
            x = s["q"][r0:r0 + n, a].double() @ k[:, a // ratio].t().contiguous() / math.sqrt(d)
            x = x.masked_fill(~see, -math.inf)
            z[:, a] = torch.logsumexp(x, -1)
            o[:, a] = torch.softmax(x, -1) @ v[:, a // ratio].contiguous()
        outs.append(o)
        lses.append(z)
        r0 += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}

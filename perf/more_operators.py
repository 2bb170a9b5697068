"""The operators of a speculative serving step on both sides of the attention over pages: norms of queries and keys with
the rotation and the append in one pass, verification of the drafted tokens, the kept tokens' rows moved together in the
pages, and requests that start from another's pages (forked) and give them back.

Head shapes are those of this repository's workloads (8 KV heads of 128 channels, 2 to 8 query heads a KV head, 36 layers)
and a few generic ones; vocabularies are generic.  Lengths, trees and paths of a case are drawn from its own `lens` seed, so
that a case is the same work whatever the seed of its values.
"""
import math

import numpy as np
import torch

own = False

FP8_MAX = 448.0
UNIT = 42                                      # probabilities are summed in units of 2^-42


# ---------------------------------------------------------------- cases

def _qkv(name, rows, q_heads, heads, dim, rotary, interleaved, norm, pool, page, strided, skip, lens):
    return {"name": name, "op": "qkv", "rows": rows, "q_heads": q_heads, "heads": heads, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "norm": norm, "pool": pool, "page": page, "strided": strided, "skip": skip, "lens": lens}


def _verify(name, batch, nodes, vocab, draft, tree, ragged, lens):
    return {"name": name, "op": "verify", "batch": batch, "nodes": nodes, "vocab": vocab, "draft": draft, "tree": tree,
            "ragged": ragged, "lens": lens}


def _compact(name, batch, nodes, context, layers, heads, dim, pool, page, lens):
    return {"name": name, "op": "compact", "batch": batch, "nodes": nodes, "context": context, "layers": layers,
            "heads": heads, "dim": dim, "pool": pool, "page": page, "lens": lens}


def _share(name, op, parents, each, tokens, layers, heads, dim, pool, page, lens):
    return {"name": name, "op": op, "parents": parents, "each": each, "tokens": tokens, "layers": layers, "heads": heads,
            "dim": dim, "pool": pool, "page": page, "lens": lens}


def listed():
    return [
        # the next tokens of 4 sequences on one layer (latency)
        _qkv("qkv 4 rows", 4, 32, 8, 128, 128, False, True, "bf16", 16, True, 0.0, 1),
        # a prompt on one layer, views of a fused projection, kept as bf16 pages
        _qkv("qkv prompt", 16384, 32, 8, 128, 128, False, True, "bf16", 16, True, 0.0, 2),
        # an odd number of rows of a padded step, rotated in part and by neighbours, rounded to an e4m3 cache
        _qkv("qkv e4m3", 5003, 16, 4, 256, 64, True, True, "e4m3", 24, False, 0.1, 3),
        # four drafted tokens of one sequence (latency)
        _verify("verify 1 x 5", 1, 5, 32000, True, False, False, 4),
        # seven drafted tokens each of a full server's sequences
        _verify("verify 64 x 8", 64, 8, 131072, True, False, False, 5),
        # trees of the likeliest tokens, drafted without probabilities, an odd vocabulary
        _verify("verify 32 trees", 32, 24, 50001, False, True, True, 6),
        # trees whose siblings were drawn from the draft's probabilities
        _verify("verify 16 drawn trees", 16, 12, 32000, True, True, True, 7),
        # kept tokens of a small batch of trees, all layers (latency)
        _compact("compact 4 x 16", 4, 16, 100, 36, 8, 128, "bf16", 16, 8),
        # kept tokens of a full server's trees, all layers
        _compact("compact 128 x 32", 128, 32, 48, 36, 8, 128, "bf16", 16, 9),
        # four answers to one prompt, all layers; they end at once
        _share("share 1 x 4", "share", 1, 4, 1000, 36, 8, 128, "bf16", 16, 10),
        # eight answers each to 32 long prompts, an e4m3 cache
        _share("share 32 x 8", "share", 32, 8, 8192, 4, 8, 64, "e4m3", 16, 11),
        # a server's requests end: prompts that others hold too, and pages of their own
        _share("release 8 x 32", "release", 8, 32, 8192, 1, 1, 64, "bf16", 16, 12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qkv", "qkv", "verify", "verify", "compact", "share", "release"])
    lens = rng.randrange(1 << 30)
    if op == "qkv":
        dim = rng.choice([64, 128, 128, 192, 256])
        heads = rng.choice([1, 2, 4, 8])
        c = _qkv("", _log_int(rng, 1, 8192), heads * rng.choice([1, 2, 4, 5, 8]), heads, dim,
                 rng.choice([dim, dim, dim // 2, 32, 0]), rng.random() < 0.3, rng.random() < 0.8,
                 rng.choice(["bf16", "e4m3"]), rng.choice([1, 8, 16, 24, 64]), rng.random() < 0.5, rng.choice([0.0, 0.2]), lens)
    elif op == "verify":
        draft, tree = rng.random() < 0.7, rng.random() < 0.5
        vocab = _log_int(rng, 1000, 40000 if draft and tree else 160000)
        batch = _log_int(rng, 1, 96)
        most = max(2, min(64, (12000000 if draft and tree else 60000000) // (batch * vocab)))
        c = _verify("", batch, _log_int(rng, 2, most), vocab, draft, tree, rng.random() < 0.5, lens)
    elif op == "compact":
        batch = _log_int(rng, 1, 128)
        c = _compact("", batch, _log_int(rng, 2, 64), _log_int(rng, 1, 96), _log_int(rng, 1, max(1, min(36, 4000 // batch))),
                     rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 192]), rng.choice(["bf16", "e4m3"]),
                     rng.choice([4, 16, 16, 24, 64]), lens)
    else:
        parents = _log_int(rng, 1, 32)
        small = op == "release"
        c = _share("", op, parents, _log_int(rng, 1, 16), _log_int(rng, 20, 8192), 1 if small else _log_int(rng, 1, 4),
                   1 if small else rng.choice([1, 2, 8]), rng.choice([64, 128]), rng.choice(["bf16", "e4m3"]),
                   rng.choice([8, 16, 16, 24, 64]), lens)
    del c["name"]
    return c


def _random(case, more=0):
    return np.random.RandomState((case["lens"] + more) % (1 << 31))


def _nodes(case):
    """Nodes of every sequence's tree (the first of them the last token that it has)."""
    n = np.full(case["batch"], case["nodes"])
    return _random(case).randint(1, case["nodes"] + 1, case["batch"]) if case.get("ragged", True) else n


def _parents(case, nodes):
    """The parent of every node, as its place in its sequence; -1 for the first."""
    r, out = _random(case, 1), []
    for n in nodes:
        if not case["tree"]:
            out.append(np.arange(n) - 1)
        else:                                  # mostly one of the last few nodes, so that trees are deep and wide
            back = np.minimum(r.randint(0, 4, n), np.maximum(np.arange(n) - 1, 0))
            out.append(np.arange(n) - 1 - back)
    return np.concatenate(out)


def _paths(case):
    """(context, nodes, kept nodes of every sequence in a row, their number)."""
    r = _random(case, 2)
    nodes, context = _nodes(case), r.randint(case["context"] // 2, case["context"] + 1, case["batch"])
    kept, lens = [], []
    for n in nodes:
        a = r.randint(0, min(n, 9))            # up to 8 accepted tokens behind the first node
        path = np.concatenate([[0], np.sort(r.choice(np.arange(1, n), a, replace=False))]) if n > 1 else np.zeros(1)
        kept.append(np.concatenate([path, np.full(n - len(path), -1)]))
        lens.append(len(path))
    return context, nodes, np.concatenate(kept).astype(np.int64), np.array(lens)


def _prompts(case):
    """Tokens of every parent."""
    return _random(case).randint(max(1, case["tokens"] // 2), case["tokens"] + 1, case["parents"])


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _kind(name):
    return torch.bfloat16 if name == "bf16" else torch.float8_e4m3fn


def _values(shape, kind, g):
    """Rows of a projection or of a cache: normal with a scale for each channel (the workloads' law)."""
    s = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    return torch.randn(shape, generator=g, device="cuda").mul_(s).to(_kind(kind))


def _pages(shape, kind, g):
    """Pages of a cache, all pools: values that are moved and never computed with, so that any bits will do."""
    n = math.prod(shape) * (2 if kind == "bf16" else 1)
    bits = torch.randint(0, 1 << 62, (-(-n // 8),), generator=g, device="cuda", dtype=torch.int64).view(torch.uint8)[:n]
    return (bits & 0x77).view(_kind(kind)).view(shape)     # (no infinities or NaN)


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def _prepare_qkv(case, g):
    rows, qh, h, d = case["rows"], case["q_heads"], case["heads"], case["dim"]
    num_pages = -(-rows // case["page"]) + 5
    pools = [_values((num_pages, case["page"], h, d), case["pool"], g) for _ in range(2)]
    if case["strided"]:                        # views of one projection's rows
        wide = _values((rows, qh + 2 * h, d), "bf16", g)
        q, k, v = wide[:, :qh], wide[:, qh:qh + h], wide[:, qh + h:]
    else:
        q, k, v = (_values((rows, n, d), "bf16", g) for n in (qh, h, h))
    slots = torch.randperm(num_pages * case["page"], generator=g, device="cuda")[:rows]
    positions = torch.randint(0, 1 << 17, (rows,), generator=g, device="cuda", dtype=torch.int32)
    pad = torch.rand(rows, generator=g, device="cuda") < case["skip"]
    norms = [(1 + 0.3 * torch.randn((1, d), generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
             for _ in range(2)]
    half = case["rotary"] // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1))
    return {"pools": pools, "q": q, "k": k, "v": v, "slots": torch.where(pad, -1, slots),
            "positions": torch.where(pad, -1, positions), "norms": norms, "freq": freq, "eps": 1e-6,
            "scale": (0.05, 0.4) if case["pool"] == "e4m3" else (1.0, 1.0),
            "q_out": torch.zeros((rows, qh, d), dtype=torch.bfloat16, device="cuda")}


def _prepare_verify(case, g):
    nodes = _nodes(case)
    parents, vocab, rows = _parents(case, nodes), case["vocab"], int(nodes.sum())
    starts = np.concatenate([[0], np.cumsum(nodes)])
    first = np.repeat(starts[:-1], nodes)
    heat = 3.0 + 3.0 * torch.rand((rows, 1), generator=g, device="cuda")
    x = torch.randn((rows, vocab), generator=g, device="cuda").mul_(heat)
    target = torch.softmax(x, -1)
    up = _ints(first + np.maximum(parents, 0), torch.int64)
    if case["draft"]:                          # the draft's own distribution behind every node, and tokens drawn from it
        draft = torch.softmax(x.add_(torch.randn((rows, vocab), generator=g, device="cuda"), alpha=0.7), -1)
        del x
        u = torch.rand((rows, 1), generator=g, device="cuda", dtype=torch.float64)
        step = max(1, (1 << 26) // vocab)
        tokens = torch.cat([(draft[up[i:i + step]].double().cumsum(-1) < u[i:i + step]).sum(-1) for i in range(0, rows, step)])
        tokens = tokens.clamp(max=vocab - 1)
    else:                                      # siblings: the target's likeliest tokens, in a mixed order
        draft = None
        del x
        best = target.topk(8, -1).indices[up]
        pick = torch.randint(0, 8, (rows, 1), generator=g, device="cuda")
        tokens = best.gather(1, pick)[:, 0]
    return {"target": target, "draft": draft, "tokens": tokens.to(torch.int32), "starts": _ints(starts),
            "parents": _ints(parents) if case["tree"] else None, "most": int(nodes.max()),
            "widest": int(np.bincount((first + parents)[parents >= 0], minlength=1).max()),      # children of a node
            "accept": torch.rand(rows, generator=g, device="cuda"), "sample": torch.rand(len(nodes), generator=g, device="cuda"),
            "kept": torch.empty(rows, dtype=torch.int32, device="cuda"),
            "kept_lens": torch.empty(len(nodes), dtype=torch.int32, device="cuda"),
            "out_tokens": torch.empty(rows, dtype=torch.int32, device="cuda")}


def _prepare_compact(case, g):
    context, nodes, kept, lens = _paths(case)
    page = case["page"]
    pages = -(-(context + nodes) // page)
    num_pages, most = int(pages.sum()) + 3, int(pages.max()) + 2
    table = torch.zeros((case["batch"], most), dtype=torch.int32, device="cuda")
    used = torch.arange(most, device="cuda")[None, :] < _ints(pages)[:, None]
    table[used] = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)[: int(pages.sum())]
    pools = _pages((2 * case["layers"], num_pages, page, case["heads"], case["dim"]), case["pool"], g)
    return {"pools": pools, "table": table, "context": _ints(context), "kept": _ints(kept), "kept_lens": _ints(lens),
            "starts": _ints(np.concatenate([[0], np.cumsum(nodes)])), "most": int(nodes.max())}


def _prepare_share(case, g):
    """Parents with their pages and rows of the table for their children; or (release) rows that stand on parents' pages,
    which more holders keep, and hold pages of their own behind them."""
    page, tokens, n = case["page"], _prompts(case), case["parents"] * case["each"]
    batch, share = case["parents"] + n, case["op"] == "share"
    held = np.zeros(batch, np.int64)
    held[: case["parents"]] = -(-tokens // page)
    whole = tokens // page
    extra_pages = _random(case, 3).randint(1, 2 + case["tokens"] // (8 * page), n)
    if not share:
        held[case["parents"]:] = np.repeat(whole, case["each"]) + extra_pages
    most = int(held.max()) + 2
    owned = int(held[: case["parents"]].sum()) + (0 if share else int(extra_pages.sum()))
    num_pages = owned + n + 9
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(most, device="cuda")[None, :]
    parent_of = np.repeat(np.arange(case["parents"]), case["each"])
    used = col < _ints(held)[:, None]
    extra = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    if not share:                              # pages of the prompts stay held by others
        common = torch.zeros((batch, most), dtype=torch.bool, device="cuda")
        common[case["parents"]:] = col < _ints(whole[parent_of])[:, None]
        used = used & ~common
    table[used] = perm[:owned]
    if not share:
        children = table[case["parents"]:]
        children[common[case["parents"]:]] = table[_ints(parent_of, torch.int64)][common[case["parents"]:]]
        extra[table[: case["parents"]][col < _ints(whole)[:, None]].long()] = 1 << 30
    free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free[: num_pages - owned] = perm[owned:]
    pools = _pages((2 * case["layers"], num_pages, page, case["heads"], case["dim"]), case["pool"], g)
    order = _random(case, 4).permutation(n)
    lens = np.zeros(batch, np.int64)
    lens[: case["parents"]] = tokens
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"pools": pools, "table": table, "held": _ints(held), "free": free, "count": _ints([num_pages - owned]),
            "extra": extra, "lens": _ints(lens), "from": _ints(parent_of[order]), "to": _ints(case["parents"] + order),
            "held_mid": torch.empty(batch, **i32), "count_mid": torch.empty(1, **i32),
            "held_out": torch.empty(batch, **i32), "count_out": torch.empty(1, **i32)}


_PREPARE = {"qkv": _prepare_qkv, "verify": _prepare_verify, "compact": _prepare_compact, "share": _prepare_share,
            "release": _prepare_share}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["case"] = case
    if own:                                    # the handles that a serving program keeps
        from entropy_coding_amd import kvc
        if case["op"] == "qkv":
            any_table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
            s["op"] = kvc.PagedQKV(kvc.PagedKV(s["pools"], any_table, case["page"]), case["q_heads"],
                                   s["freq"] if case["rotary"] else None, *s["norms"], eps=s["eps"],
                                   interleaved=case["interleaved"], k_scale=s["scale"][0], v_scale=s["scale"][1])
        elif case["op"] == "verify":
            s["op"] = kvc.DraftVerifier(case["batch"], case["vocab"], len(s["tokens"]))
        elif case["op"] == "compact":
            s["op"] = kvc.PagedCompaction(kvc.PagedKV(s["pools"].unbind(0), s["table"], case["page"]))
        else:
            paged = kvc.PagedKV(s["pools"].unbind(0), s["table"], case["page"])
            if case["op"] == "share":
                s["forks"] = kvc.SharedPages(paged, s["held"], s["free"], s["count"], s["extra"], held_out=s["held_mid"],
                                             free_count_out=s["count_mid"])
                s["ends"] = kvc.SharedPages(paged, s["held_mid"], s["free"], s["count_mid"], s["extra"],
                                            held_out=s["held_out"], free_count_out=s["count_out"])
            else:
                s["ends"] = kvc.SharedPages(paged, s["held"], s["free"], s["count"], s["extra"], held_out=s["held_out"],
                                            free_count_out=s["count_out"])
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_norm(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w[0].float()


def _plain_rotate(x, s, case):
    n = case["rotary"]
    if n == 0:
        return x
    turn = s["positions"].double()[:, None, None] * s["freq"]
    c, z = turn.cos().float(), turn.sin().float()
    pairs = x[..., :n].unflatten(-1, (n // 2, 2)) if case["interleaved"] else x[..., :n].unflatten(-1, (2, n // 2)).transpose(-1, -2)
    a, b = pairs[..., 0], pairs[..., 1]
    y = torch.stack([a * c - b * z, a * z + b * c], -1)
    y = y if case["interleaved"] else y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., n:]], -1)


def _plain_qkv(s, case):
    h, d = case["heads"], case["dim"]
    q, k = (_plain_rotate(_plain_norm(x, w, s["eps"]), s, case) for x, w in zip((s["q"], s["k"]), s["norms"]))
    there = (s["positions"] >= 0)[:, None, None]
    s["q_out"].copy_(torch.where(there, q.to(torch.bfloat16), s["q_out"]))
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    for pool, x, scale in zip(s["pools"], (k, s["v"].float()), s["scale"]):
        x = x[keep]
        if pool.element_size() == 1:
            x = (x / scale).clamp(-FP8_MAX, FP8_MAX)
        bits = torch.int16 if pool.element_size() == 2 else torch.uint8
        pool.view(bits).view(-1, h, d)[at] = x.to(pool.dtype).view(bits)


def _units(y):
    return (y.double() * 2.0 ** UNIT).long()


def _plain_verify(s, case):
    """Every node is tested as if its parent were reached and its siblings before it rejected; which ones are in fact
    follows from these tests alone."""
    batch, n, vocab = case["batch"], s["most"], case["vocab"]
    starts = s["starts"].long()
    i = torch.arange(n, device="cuda")
    real = starts[:-1, None] + i < starts[1:, None]
    row = torch.where(real, starts[:-1, None] + i, 0)                                      # [batch, n]
    parent = torch.where(real & (i > 0), (i - 1).expand(batch, n) if s["parents"] is None else s["parents"].long()[row], -1)
    up = torch.where(parent >= 0, starts[:-1, None] + parent, 0)
    token, u = s["tokens"].long()[row], s["accept"].double()[row]
    before = (parent[:, :, None] == parent[:, None, :]) & (i[None, :] < i[:, None]) & (parent >= 0)[:, :, None]
    rank = before.sum(-1)
    p, q = s["target"], s["draft"]
    if q is None:
        again = (before & (token[:, :, None] == token[:, None, :])).any(-1)                # a token that was rejected has no mass left
        y = torch.where(again, 0.0, p[up, token])
        mass = ((1 << UNIT) - torch.where(before, _units(y)[:, None, :], 0).sum(-1)).clamp(min=0)
        ok = u * mass.double() < y.double() * 2.0 ** UNIT
    else:
        ok = u * q[up, token].double() < p[up, token].double()
        y = p
        for r in range(1, s["widest"]):        # the r-th sibling meets what r rejections left
            y = (y - q).clamp(min=0)
            z = _units(y).sum(-1, keepdim=True)
            y = y * torch.where(z > 0, 2.0 ** UNIT / z.double(), 0.0).float()
            ok = torch.where(rank == r, u * q[up, token].double() < y[up, token].double(), ok)
    ok = ok & (parent >= 0)
    reached = torch.where(i == 0, real, ok & ~(before & ok[:, None, :]).any(-1))
    at = parent.clamp(min=0)
    for _ in range(max(1, math.ceil(math.log2(n)))):                                       # ... and so are all nodes above
        reached = reached & reached.gather(1, at)
        at = at.gather(1, at)
    lens = reached.sum(-1)
    order = torch.where(reached, i, n).sort(-1).values
    stop = torch.where(reached, i, 0).amax(-1)
    last = starts[:-1] + stop
    some = real[:, 0]
    last = torch.where(some, last, 0)
    tried = (parent == stop[:, None]) & real & (i > 0)
    y = whole = p[last]
    if q is None:
        y = torch.cat([y, y.new_zeros(batch, 1)], 1).scatter(1, torch.where(tried, token, vocab), 0.0)[:, :vocab]
    else:
        left = q[last]
        for r in range(s["widest"]):
            z = _units(y).sum(-1, keepdim=True)
            scale = torch.where(z > 0, 2.0 ** UNIT / z.double(), 0.0).float() if r else 1.0
            y = torch.where(r < tried.sum(-1, keepdim=True), (y * scale - left).clamp(min=0), y)
    y = torch.where(_units(y).sum(-1, keepdim=True) > 0, y, whole)
    upto = _units(y).cumsum(-1)
    total = upto[:, -1:]
    point = torch.minimum((s["sample"].double()[:, None] * total.double()).long(), total - 1)
    drawn = (upto <= point).sum(-1)
    kept = torch.where(order < n, order, -1)
    out = torch.where(i < lens[:, None] - 1, token.gather(1, torch.roll(kept, -1, 1).clamp(min=0)),
                      torch.where(i == lens[:, None] - 1, drawn[:, None], -1))
    s["kept"].copy_(kept[real])
    s["kept_lens"].copy_(lens)
    s["out_tokens"].copy_(out[real])


def _plain_compact(s, case):
    page, starts = case["page"], s["starts"].long()
    j = torch.arange(s["most"], device="cuda")
    go = j < s["kept_lens"][:, None]
    node = s["kept"].long()[torch.where(go, starts[:-1, None] + j, 0)]
    table, context = s["table"].long(), s["context"].long()[:, None]
    from_, to = ((table.gather(1, torch.where(go, t, 0) // page) * page + t % page)[go] for t in (context + node, context + j))
    flat = s["pools"].view(torch.int16 if case["pool"] == "bf16" else torch.uint8).flatten(1, 2)
    flat[:, to] = flat[:, from_]


def _plain_fork(s, case):
    page, table = case["page"], s["table"]
    parent, child = s["from"].long(), s["to"].long()
    length = s["lens"].long()[parent]
    whole, rest = length // page, length % page
    tail = (rest > 0).long()
    place = s["count"].long() - 1 - (tail.cumsum(0) - tail)
    new = s["free"][place]
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    shared = col < whole[:, None]
    last = table[parent].gather(1, whole[:, None].clamp(max=table.shape[1] - 1))[:, 0]
    mine = torch.where((col == whole[:, None]) & (tail > 0)[:, None], new[:, None], table[child])
    table[child] = torch.where(shared, table[parent], mine)
    pages = table[parent][shared].long()
    s["extra"].index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    s["held_mid"].copy_(s["held"].index_copy(0, child, (whole + tail).int()))
    s["count_mid"].copy_(s["count"] - tail.sum())
    pools = s["pools"].view(torch.int16 if case["pool"] == "bf16" else torch.uint8)
    row = torch.arange(page, device="cuda")
    copied = (row[None, :] < rest[:, None])
    b, r = copied.nonzero(as_tuple=True)
    pools[:, new.long()[b], r] = pools[:, last.long()[b], r]


def _plain_release(s, case, rows, held, count):
    table = s["table"]
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    pages = table[rows][col < held[rows][:, None]].long()
    leaves = torch.bincount(pages, minlength=len(s["extra"]))
    freed = leaves > s["extra"]
    s["extra"].copy_((s["extra"] - leaves).clamp(min=0))
    page = freed.nonzero()[:, 0].int()
    s["free"][count.long() + torch.arange(len(page), device="cuda")] = page
    s["held_out"].copy_(held.index_fill(0, rows, 0))
    s["count_out"].copy_(count + len(page))


def run(state):
    s, case = state, state["case"]
    if case["op"] == "qkv":
        if own:
            s["op"](0, s["q"], s["k"], s["v"], s["slots"], s["positions"], out=s["q_out"])
        else:
            _plain_qkv(s, case)
        return {"q": s["q_out"], "k": s["pools"][0], "v": s["pools"][1]}
    if case["op"] == "verify":
        if own:
            s["op"](s["target"], s["tokens"], s["starts"], s["accept"], s["sample"], parents=s["parents"], draft=s["draft"],
                    kept=s["kept"], kept_lens=s["kept_lens"], out_tokens=s["out_tokens"])
        else:
            _plain_verify(s, case)
        return {k: s[k] for k in ("kept", "kept_lens", "out_tokens")}
    if case["op"] == "compact":
        if own:
            s["op"](s["starts"], s["context"], s["kept"], s["kept_lens"])
        else:
            _plain_compact(s, case)
        return {"pools": s["pools"]}
    if case["op"] == "share":
        if own:
            s["forks"].fork(s["from"], s["to"], s["lens"])
            s["ends"].release(s["to"])
        else:
            _plain_fork(s, case)
            _plain_release(s, case, s["to"].long(), s["held_mid"], s["count_mid"])
        return {k: s[k] for k in ("pools", "table", "held_mid", "count_mid", "held_out", "count_out", "free", "extra")}
    if own:
        s["ends"].release(s["to"])
    else:
        _plain_release(s, case, s["to"].long(), s["held"], s["count"])
    return {k: s[k] for k in ("held_out", "count_out", "free", "extra")}


# ---------------------------------------------------------------- work and the 64-bit values

def work(case):
    size = 2 if case.get("pool") == "bf16" else 1
    if case["op"] == "qkv":
        rows, qh, h, d = case["rows"] * (1.0 - case["skip"]), case["q_heads"], case["heads"], case["dim"]
        return {"bytes": rows * d * (4 * qh + 2 * h * (2 + size)) + 12 * case["rows"] + 4 * case["rotary"] + 4 * d,
                "flops": rows * (qh + h) * (4 * d * case["norm"] + 3 * case["rotary"])}
    if case["op"] == "verify":
        # the distribution (or two) that each sequence's last token is drawn from, and a few values a node
        rows = int(_nodes(case).sum())
        return {"bytes": case["batch"] * case["vocab"] * (8 if case["draft"] else 4) + rows * (28 if case["draft"] else 24),
                "flops": 3.0 * case["batch"] * case["vocab"]}
    row = case["heads"] * case["dim"] * size * 2 * case["layers"]
    if case["op"] == "compact":
        context, nodes, kept, lens = _paths(case)
        starts = np.concatenate([[0], np.cumsum(nodes)])
        moved = sum(int((kept[a:a + n] != np.arange(n)).sum()) for a, n in zip(starts, lens))
        return {"bytes": 2.0 * moved * row + 4 * int(lens.sum()) + 12 * case["batch"] + 8 * moved, "flops": 0}
    tokens = _prompts(case)
    whole, rest, page = tokens // case["page"], tokens % case["page"], case["page"]
    n, each = case["parents"] * case["each"], case["each"]
    if case["op"] == "share":
        # rows of the unfilled pages read once a parent and written once a child; a page number read and written and a
        # count raised and lowered for each shared page, and one page number pushed for each copied one
        copied = float(rest.sum()) * row * (1 + each)
        return {"bytes": copied + float(whole.sum()) * each * (8 + 4) + float(whole.sum()) * 16 + 16.0 * n, "flops": 0}
    mine = _random(case, 3).randint(1, 2 + case["tokens"] // (8 * page), n)
    return {"bytes": 4.0 * (float(whole.sum()) * each + mine.sum()) + 8.0 * float(whole.sum()) + 8.0 * mine.sum() + 12.0 * n,
            "flops": 0}


def exact(case, seed):
    g = _gen(seed)
    if case["op"] == "qkv":
        s = _prepare_qkv(case, g)
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        half, d = case["rotary"] // 2, case["dim"]
        a, b = (2 * torch.arange(half), 2 * torch.arange(half) + 1) if case["interleaved"] else (torch.arange(half), half + torch.arange(half))
        out = []
        for x, w in zip((s["q"], s["k"]), s["norms"]):
            y = x[keep].double()
            if w is not None:
                y = y / ((y ** 2).sum(-1, keepdim=True) / d + s["eps"]).sqrt() * w.double()
            angle = torch.outer(s["positions"][keep].double(), s["freq"])[:, None]
            turned = y.clone()
            turned[..., a.cuda()] = y[..., a.cuda()] * angle.cos() - y[..., b.cuda()] * angle.sin()
            turned[..., b.cuda()] = y[..., a.cuda()] * angle.sin() + y[..., b.cuda()] * angle.cos()
            out.append(turned)
        q = s["q_out"].double()
        q[keep] = out[0]
        pools = []
        for pool, x, scale in zip(s["pools"], (out[1], s["v"][keep].double()), s["scale"]):
            y = pool.double().view(-1, case["heads"], d)
            y[s["slots"][keep]] = (x / scale).clamp(-FP8_MAX, FP8_MAX) if case["pool"] == "e4m3" else x
            pools.append(y.view(pool.shape))
        return {"q": q, "k": pools[0], "v": pools[1]}
    if case["op"] in ("verify", "release"):
        return None                            # whole numbers: the plain form's have to be met
    if case["op"] == "compact":
        s = _prepare_compact(case, g)
        pools = s["pools"].double()
        context, nodes, kept, lens = _paths(case)
        table, page, r0 = s["table"].cpu().numpy(), case["page"], 0
        for b in range(case["batch"]):
            for j in range(lens[b]):           # in order, each row read before a later one is written over it
                x, y = int(context[b] + kept[r0 + j]), int(context[b] + j)
                if x != y:
                    pools[:, table[b, y // page], y % page] = pools[:, table[b, x // page], x % page]
            r0 += nodes[b]
        return {"pools": pools}
    s = _prepare_share(case, g)
    pools, page = s["pools"].double(), case["page"]
    table, free, at = s["table"].cpu().numpy(), s["free"].cpu().numpy(), int(s["count"])
    for parent, n in zip(s["from"].tolist(), s["lens"].cpu().numpy()[s["from"].cpu().numpy()].tolist()):
        if n % page:
            at -= 1
            pools[:, free[at], : n % page] = pools[:, table[parent, n // page], : n % page]
    return {"pools": pools, "table": None, "held_mid": None, "count_mid": None, "held_out": None, "count_out": None,
            "free": None, "extra": None}

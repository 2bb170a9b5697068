"""Plain forms of the paged-cache operators for the tests: loops and float64,
written from the operators' definitions."""
import numpy as np
import torch


def block_table(table, held, free, count, page, cached, new, max_rows, trim):
    """One step on copies: (table, held, free, count, row_starts, slots, positions)."""
    table, held, free = table.copy(), held.copy(), free.copy()
    batch = table.shape[0]
    need = [-(-(int(c) + int(n)) // page) for c, n in zip(cached, new)]
    if trim:
        back = [table[b, j] for b in range(batch) for j in range(need[b], held[b])]
        for p in reversed(back):
            free[count] = p
            count += 1
    for b in range(batch):
        for j in range(held[b], need[b]):
            count -= 1
            table[b, j] = free[count]
        held[b] = need[b] if trim else max(held[b], need[b])
    starts, slots, positions = [0], [], []
    for b in range(batch):
        for i in range(int(new[b])):
            pos = int(cached[b]) + i
            slots.append(int(table[b, pos // page]) * page + pos % page)
            positions.append(pos)
        starts.append(len(slots))
    pad = max_rows - len(slots)
    return (table, held, free, count, np.array(starts, np.int32), np.array(slots + [-1] * pad, np.int64),
            np.array(positions + [-1] * pad, np.int32))


def seen(context, nodes, mask, chain_row):
    """Which of context + nodes tokens a row sees: bits of its mask (a list of
    64-bit words), or (mask None) the chain up to drafted token chain_row."""
    see = np.zeros(context + nodes, bool)
    see[:context] = True
    for j in range(nodes):
        if mask is None:
            see[context + j] = j <= chain_row
        elif j // 64 < len(mask):
            see[context + j] = bool((int(mask[j // 64]) >> (j % 64)) & 1)
    return see


def attention(pool_k, pool_v, table, page, q, starts, contexts, mask, scale, v_scale):
    """float64 out [rows, q_heads, D], lse, and for each output a bound on its
    error: `loose` the sum of p |v| / l (what a relative error of the weights
    is multiplied with) and `score` the largest sum of |q k| x |scale|."""
    rows, q_heads, d = q.shape
    heads = pool_k.shape[2]
    ratio = q_heads // heads
    out = np.zeros((rows, q_heads, d))
    lse = np.full((rows, q_heads), -np.inf)
    loose, score = np.zeros((rows, q_heads, d)), np.zeros((rows, q_heads))
    k_all = pool_k.reshape(-1, heads, d)
    v_all = pool_v.reshape(-1, heads, d)
    for b in range(len(starts) - 1):
        n, c = int(starts[b + 1] - starts[b]), int(contexts[b])
        if n == 0:
            continue
        t = np.arange(c + n)
        slot = table[b, t // page].astype(np.int64) * page + t % page
        see = np.stack([seen(c, n, None if mask is None else mask[starts[b] + i], i) for i in range(n)])
        for h in range(heads):
            k, v = k_all[slot, h], v_all[slot, h]
            for i in range(n):
                w = see[i]
                if not w.any():
                    continue
                for g in range(ratio):
                    a = h * ratio + g
                    x = q[starts[b] + i, a]
                    s = k[w] @ x * scale
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    out[starts[b] + i, a] = v_scale * (p @ v[w]) / total
                    lse[starts[b] + i, a] = m + np.log(total)
                    loose[starts[b] + i, a] = v_scale * (p @ np.abs(v[w])) / total
                    score[starts[b] + i, a] = np.abs(scale) * (np.abs(k[w]) @ np.abs(x)).max()
    return out, lse, loose, score


def tolerances(out, loose, score, tokens, d, weight_step=2.0 ** -8):
    """Bounds on |kernel - float64| for out and lse.  A score sums d products
    in float32 (d steps of 2^-24 of the sum of |q k|), is scaled (two
    roundings) and goes through an exponential good to 2 units in the last
    place and the difference to the maximum (one rounding of a value up to
    2 x score in units of log 2): `s`.  Weights are rounded to bf16
    (weight_step) and summed with V in float32 over `tokens` terms; so is l.
    The quotient, the scale and the output's bf16 are one rounding each."""
    s = (d + 8) * 2.0 ** -24 * score + 4 * 2.0 ** -23
    sums = (tokens + 16) * 2.0 ** -24
    rel = s + sums
    tol_out = 2.0 ** -8 * np.abs(out) + (2 * rel + weight_step)[..., None] * loose * (1 + 2.0 ** -8) + 2.0 ** -133
    tol_lse = rel + 2.0 ** -22 * (score + np.log(tokens + 1.0) + 1.0)
    return tol_out, tol_lse


def tree(nodes, words, rng):
    """Mask words [sum of nodes, words] (int64) of random trees: a node sees
    itself and its ancestors."""
    rows = []
    for n in nodes:
        see = []
        for i in range(int(n)):
            own = 1 << i
            see.append(own | (see[rng.integers(0, i)] if i else 0))
        for m in see:
            w = [(m >> (64 * k)) & (2 ** 64 - 1) for k in range(words)]
            rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in w])
    return np.array(rows, np.int64).reshape(-1, words)


def to_f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().float().double().numpy()

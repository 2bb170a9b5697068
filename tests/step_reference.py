"""Plain forms of the speculative step's operators for the tests: loops,
float64 and whole numbers, written from the operators' definitions."""
import numpy as np
import torch

BF16_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -4      # half a step, relative to the value
BF16_LEAST, E4M3_LEAST = 2.0 ** -134, 2.0 ** -10  # ... and among the subnormal numbers


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def norm_rotate(x, weight, eps, positions, frequencies, neighbours):
    """(values, size): x [rows, heads, channels] normed (weight or None) and
    rotated in float64, and for each value the sum of magnitudes that float32
    errors of the norm and the angle's functions scale with."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    size, half = np.abs(y), len(frequencies)
    if half == 0:
        return y, size
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, half + i)
    t = positions[:, None, None].astype(np.float64) * frequencies
    out = y.copy()
    out[..., a] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t)
    out[..., b] = y[..., a] * np.sin(t) + y[..., b] * np.cos(t)
    both = (np.abs(y[..., a]) + np.abs(y[..., b])) * (1 + np.abs(t) * 2.0 ** -32)
    size = size.copy()
    size[..., a] = size[..., b] = both
    return out, size


# Errors of the float32 computation before the last rounding, relative to
# `size`: 16 products and 16 lanes summed (20 roundings of 2^-24, half of it
# through the root), the root 2^-23, two products of 2^-24: under 2^-20; sine
# and cosine: the turn's rounding 2^-25 x 2 pi and two units of 2^-24: under
# 2^-21; the rotation's own two roundings 2^-23.  Of the angle in float64:
# three roundings (by 2 pi, by the position, and the reference's own), each
# 2^-53 of the angle: 2^-51 of it, which is `size`'s 2^-32 times this.
FLOAT_ERROR = 2.0 ** -19


def tolerance_bf16(y, size):
    e = size * FLOAT_ERROR
    return BF16_HALF * (np.abs(y) + e) + e + BF16_LEAST


def tolerance_e4m3(z, size):
    """z: the quotient by the scale; size likewise."""
    e = size * FLOAT_ERROR + np.abs(z) * 2.0 ** -24
    return np.maximum(E4M3_HALF * (np.abs(z) + e), E4M3_LEAST) + e


# ---------------------------------------------------------------- verification

UNIT = 2.0 ** 42


def clean(p):
    """Probabilities as they count: float32 in [0, 1], NaN as 0."""
    return np.clip(np.where(np.isnan(p), np.float32(0), p), np.float32(0), np.float32(1)).astype(np.float32)


def units(y):
    return np.floor(y.astype(np.float64) * UNIT).astype(np.int64)


def verify(starts, tokens, parents, target, draft, accept, sample):
    """Per sequence (kept places, new tokens), walked node by node."""
    out = []
    for b in range(len(starts) - 1):
        s, n = int(starts[b]), int(starts[b + 1] - starts[b])
        if n <= 0 or s < 0 or s + n > len(tokens) or n > 1024:
            out.append(([], []))
            continue
        path, y, rejected, mass = [0], clean(target[s]), 0, 1 << 42
        for i in range(1, n):
            if (i - 1 if parents is None else parents[s + i]) != path[-1]:
                continue
            t, u = int(tokens[s + i]), np.float64(accept[s + i])
            there = 0 <= t < len(y)
            if draft is not None:
                q = clean(draft[s + path[-1]])
                if rejected:
                    z = int(units(y).sum())
                    y = y * (np.float32(UNIT / np.float64(z)) if z else np.float32(0))
                ok = there and u * np.float64(q[t]) < np.float64(y[t])
                if not ok:
                    y = np.maximum(y - q, np.float32(0))
            else:
                ok = there and u * np.float64(mass) < np.float64(y[t]) * UNIT
                if not ok and there:
                    mass = max(0, mass - int(units(y[t])))
                    y = y.copy()
                    y[t] = 0
            rejected += 1
            if ok:
                path, y, rejected, mass = path + [i], clean(target[s + i]), 0, 1 << 42
        if units(y).sum() == 0:
            y = clean(target[s + path[-1]])
        upto = np.cumsum(units(y))
        total = int(upto[-1])
        u = float(sample[b])
        point = min(int(u * float(total)) if u > 0 else 0, total - 1)
        last = int((upto <= point).sum()) if total else -1
        out.append((path, [int(tokens[s + i]) for i in path[1:]] + [last]))
    return out


# ---------------------------------------------------------------- pages

def compact(pools, table, page, starts, contexts, kept, lens):
    """pools [n, pages, page, ...] on the host, in place."""
    for b in range(len(lens)):
        for j in range(int(lens[b])):
            x, y = int(contexts[b] + kept[starts[b] + j]), int(contexts[b] + j)
            if x != y:
                pools[:, table[b, y // page], y % page] = pools[:, table[b, x // page], x % page]


def fork(pools, table, held, free, count, extra, page, parents, children, lens):
    """On copies (pools in place): (table, held, count, extra)."""
    table, held, extra = table.copy(), held.copy(), extra.copy()
    for p, c in zip(parents, children):
        if c == -1:
            continue
        whole, rest = divmod(int(lens[p]), page)
        table[c, :whole] = table[p, :whole]
        for j in range(whole):
            extra[table[p, j]] += 1
        if rest:
            count -= 1
            table[c, whole] = free[count]
            pools[:, free[count], :rest] = pools[:, table[p, whole], :rest]
        held[c] = whole + (rest > 0)
    return table, held, count, extra


def release(table, held, free, count, extra, requests):
    """On copies: (held, free, count, extra)."""
    held, free, extra = held.copy(), free.copy(), extra.copy()
    gone = []
    for r in requests:
        if r == -1:
            continue
        for j in range(held[r]):
            page = table[r, j]
            if extra[page] == 0:
                gone.append(page)
            else:
                extra[page] -= 1
        held[r] = 0
    for page in sorted(gone):
        free[count] = page
        count += 1
    return held, free, count, extra

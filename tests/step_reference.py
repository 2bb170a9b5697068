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

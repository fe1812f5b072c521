"""The rotation and the 4-bit cache on the CPU, in float64 from their
definitions: numbers are rounded by looking for the nearest of all that the
format has.  Test infrastructure, sharing no code with the GPU path.
"""
from __future__ import annotations

import numpy as np

from . import paged

GROUP = 16
FOURS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])                 # e2m1
EIGHTS = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                   for e in range(16) for m in range(8)][:127])    # e4m3; 127 is NaN
NAN_SCALE = 127


def nearest(y, numbers):
    """Indexes of the numbers nearest to y >= 0, of two equally near the even
    one; the largest for what is past it."""
    high = np.clip(np.searchsorted(numbers, y), 1, len(numbers) - 1)
    below, above = y - numbers[high - 1], numbers[high] - y
    up = (above < below) | ((above == below) & (high % 2 == 0))
    return np.where(up, high, high - 1)


def encode(x, gain=1.0):
    """(codes [..., D / 2], scales [..., D / 16]) as uint8, of x [..., D]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    top = np.abs(g).max(-1)
    sound = np.isfinite(top)
    scale = np.where(sound, nearest(np.where(sound, top, 0) / (6 * gain), EIGHTS), NAN_SCALE)
    unit = np.where(sound, np.append(EIGHTS, 0)[scale] * gain, 0)[..., None]
    with np.errstate(invalid="ignore"):
        code = nearest(np.where(unit > 0, np.abs(g) / np.where(unit > 0, unit, 1), 0), FOURS)
    code = np.where(unit > 0, code + 8 * np.signbit(g), 0).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.astype(np.uint8)


def decode(codes, scales, gain=1.0):
    """Values [..., D] of codes and scales as uint8."""
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    values = np.concatenate([FOURS, -FOURS])[both]
    return values * np.repeat(np.append(EIGHTS, np.nan)[scales & 127] * np.where(scales > 127, -1, 1), GROUP, -1) * gain


def rotate(x, positions, table, interleaved=False):
    """x [T, heads, D] turned by the rows `positions` of table [n, rot]; zeros
    where there is no position."""
    y = np.zeros_like(x)
    rot = table.shape[1]
    for t, p in enumerate(positions):
        if not 0 <= p < len(table):
            continue
        y[t] = x[t]
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = table[p, i], table[p, rot // 2 + i]
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return y


def rotation_tolerance(x, y, positions, table, dtype, interleaved=False):
    """Bound of a rotated value's error: two float32 products and their
    difference, each within 2^-24 of |x cos| + |y sin|, and one rounding."""
    u, tiny = paged.UNIT[dtype]
    terms = rotate(np.abs(x), positions, np.abs(table), interleaved)   # |x sin| + |y cos| where the sum is
    sums = np.abs(terms)
    for t, p in enumerate(positions):
        if 0 <= p < len(table):
            for i in range(table.shape[1] // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + table.shape[1] // 2)
                sums[t, :, a] = np.abs(x[t, :, a] * table[p, i]) + np.abs(x[t, :, b] * table[p, table.shape[1] // 2 + i])
    off = 3 * 2.0 ** -24 * sums
    return u * (np.abs(y) + off) + off + tiny


def attention(q, k, v, cu_new, kv_len, scale, dtype):
    """paged.attention over one page [1, Hk, L, D] of the values that the cache
    holds.  The operands of both products are float16, in which those values
    are exact; the result is rounded once to `dtype`."""
    r = paged.attention(q, k, v, np.zeros((1, 1), int), cu_new, kv_len, scale, "f16")
    return r._replace(out_tol=r.out_tol + (paged.UNIT["bf16"][0] * np.abs(r.out) if dtype == "bf16" else 0))

"""Head norms and rotation, a cache's quantization, and attention, in fp64 (test infrastructure).

``attend`` returns besides the outputs what the tests' tolerances are made of: for every output the sum of p |v| and the
root of the sum of (p v)^2 over the keys (p: the probabilities), and for every row the largest sum of |q k| of a key it
sees.
"""

import numpy as np

from . import f8


def heads(x, weight, eps, positions, inv_freq, interleaved):
    """x [T, heads, D] normed (weight None: not) and rotated (inv_freq None: not); also the largest magnitude that each
    output is made of."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    size = np.abs(y)
    if inv_freq is not None:
        n = len(inv_freq)
        first = 2 * np.arange(n) if interleaved else np.arange(n)
        second = first + (1 if interleaved else n)
        t = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
        c, s = np.cos(t), np.sin(t)
        a, b = y[..., first].copy(), y[..., second].copy()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size


def quantize(x):
    """x [..., D] -> e4m3 codes uint8 and fp32 scales [...], one a row."""
    x = np.asarray(x, dtype=np.float64)
    s = f8.scale(np.abs(x).max(-1))
    with np.errstate(invalid="ignore"):
        return f8.encode(x / s.astype(np.float64)[..., None]), s


def values(codes, scales):
    return f8.e4m3_values()[codes] * np.asarray(scales, dtype=np.float64)[..., None]


def attend(q, k, v, scale, seen):
    """One head: q [n, D], k and v [m, D], seen [n, m] -> outputs [n, D] (zeros where a row sees nothing), and the parts of a
    tolerance.  Keys and values that a row does not see take no part, whatever they hold."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    n, m = seen.shape
    out, spread, noise, reach = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q), np.zeros((n, 1))
    for i in range(n):
        j = np.flatnonzero(seen[i])
        if not len(j):
            continue
        s = scale * (k[j] @ q[i])
        p = np.exp(s - s.max())
        p /= p.sum()
        out[i] = p @ v[j]
        spread[i] = p @ np.abs(v[j])
        noise[i] = np.sqrt((p * p) @ (v[j] * v[j]))
        reach[i] = scale * (np.abs(k[j]) @ np.abs(q[i])).max()
    return out, spread, noise, reach


def causal(n, m):
    """seen [n, m] of the last n of m tokens."""
    return np.arange(m)[None] <= np.arange(n)[:, None] + (m - n)

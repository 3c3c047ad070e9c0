"""e4m3 values with one scale per block of 128, and the products of two such operands, in fp64 (test infrastructure).

Definition: a block's scale is s = max(fp32(max|v| / 448), 2^-80), NaN when the block holds an Inf or a NaN; a code is
the e4m3 value nearest to the real quotient v / s, ties to the even mantissa.  e4m3: sign, 4 exponent bits (bias 7), 3
mantissa bits; exponent 0 is subnormal (steps of 2^-9), the all-ones code is NaN, the largest value 448.
"""

import numpy as np

BLOCK = 128
MIN_SCALE = 2.0 ** -80


def padded(n):
    return -(-n // BLOCK) * BLOCK


def e4m3_values():
    """The 256 codes' values, fp64 (NaN for 0x7F and 0xFF)."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        out[c] = sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    out[[0x7F, 0xFF]] = np.nan
    return out


def encode(v):
    """Nearest e4m3 codes of fp64 v with |v| <= 448 (ties to even; NaN gives 0x7F), uint8."""
    v = np.asarray(v, dtype=np.float64)
    grid = e4m3_values()[:127]
    middle = (grid[1:] + grid[:-1]) / 2
    a = np.abs(v)
    n = np.searchsorted(middle, a)              # middles strictly below a
    tie = (n < 126) & (middle[np.minimum(n, 125)] == a)
    n = n + (tie & (n % 2 == 1))
    code = n.astype(np.uint8) | np.where(np.signbit(v), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(v), np.uint8(0x7F), code)


def scale(block_max):
    """fp32 scales of blocks whose largest magnitudes are given (NaN or Inf: NaN)."""
    m = np.asarray(block_max, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        s = np.maximum((m / 448.0).astype(np.float32), np.float32(MIN_SCALE))
    return np.where(np.isfinite(m), s, np.float32(np.nan)).astype(np.float32)


def quantize_rows(x):
    """x [R, C] -> codes uint8 [R, padded C], scales fp32 [padded C / 128, R]."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    full = np.zeros((R, padded(C)))
    full[:, :C] = x
    g = full.reshape(R, -1, BLOCK)
    s = scale(np.abs(g).max(axis=2))
    with np.errstate(invalid="ignore"):
        codes = encode(g / s.astype(np.float64)[:, :, None])
    return codes.reshape(R, -1), np.ascontiguousarray(s.T)


def quantize_weight(w):
    """w [M, K] -> codes uint8 [M, padded K], scales fp32 [padded M / 128, padded K / 128]."""
    w = np.asarray(w, dtype=np.float64)
    M, K = w.shape
    full = np.zeros((padded(M), padded(K)))
    full[:M, :K] = w
    b = full.reshape(padded(M) // BLOCK, BLOCK, padded(K) // BLOCK, BLOCK)
    s = scale(np.abs(b).max(axis=(1, 3)))
    with np.errstate(invalid="ignore"):
        codes = encode(b / s.astype(np.float64)[:, None, :, None])
    return codes.reshape(padded(M), -1)[:M], s


def rows_values(codes, scales, C):
    """What quantize_rows' output stands for, fp64 [R, C]."""
    v = e4m3_values()[codes].reshape(codes.shape[0], -1, BLOCK)
    return (v * scales.T.astype(np.float64)[:, :, None]).reshape(codes.shape[0], -1)[:, :C]


def weight_values(codes, scales, K):
    """What quantize_weight's output stands for, fp64 [M, K]."""
    M = codes.shape[0]
    full = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0)[:M], BLOCK, 1)
    return (e4m3_values()[codes] * full)[:, :K]


def product_bound(xv, wv, f8_cores=False):
    """|y - exact| allowed for an fp32 product over values xv [N, K], wv [M, K], before y's own rounding: 128 terms of a
    group summed with a step's error each (2^-23, rounded or cut), a rounding of the product with a scale (or of the scales'), one per
    group's fma and one per partial sum that is joined (at most 16).  f8_cores: the matrix cores also drop what is below
    2^-13 of the largest of 8 products' exponents, at most 8 * 2^-13 of that largest product."""
    groups = padded(xv.shape[1]) // BLOCK
    step = BLOCK * 2.0 ** -23 + (groups + 2 + 16) * 2.0 ** -24 + (2.0 ** -10 if f8_cores else 0.0)
    return (np.abs(xv) @ np.abs(wv).T) * step

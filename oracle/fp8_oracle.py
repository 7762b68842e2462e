"""Float64 reference of 8-bit floats (e4m3) with a scale for each block of 128,
and of their products.

A code's bit 7 is the sign, bits 3-6 the exponent (bias 7, 0: steps of 2^-9),
bits 0-2 the mantissa; 0x7F and 0xFF are NaN.  Written from the format's
definition: codes are found among all values by their midpoints.
"""
from __future__ import annotations

import numpy as np

FP8_BLOCK = 128
FP8_MAX = 448.0


def _value(code: int) -> float:
    e, m = (code >> 3) & 15, code & 7
    if code & 127 == 127:
        return float("nan")
    v = np.ldexp(m, -9) if e == 0 else np.ldexp(8 + m, e - 10)
    return float(-v if code & 128 else v)


FP8_VALUES = np.array([_value(c) for c in range(256)])
_MIDS = (FP8_VALUES[1:127] + FP8_VALUES[:126]) / 2          # between codes c and c + 1


def fp8_blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def fp8_nearest_code(v):
    """Codes of the values nearest to v (float64), ties to the even code, the
    code of 448 for everything beyond."""
    a = np.abs(v)
    c = np.searchsorted(_MIDS, a, side="left")               # a midpoint itself: the lower code
    tie = (c < 126) & (a == _MIDS[np.minimum(c, 125)]) & (c % 2 == 1)
    return np.where(tie, c + 1, c) | np.where(np.signbit(v), 128, 0)


def fp8_spread(scales, block_rows: int, m: int, n: int):
    """Scales of every element of an m x n matrix, float64."""
    s = np.repeat(np.asarray(scales, dtype=np.float64), FP8_BLOCK, axis=1)[:, :n]
    return np.repeat(s, block_rows, axis=0)[:m]


def fp8_quantize(W, block_rows: int):
    """(codes m x n, float32 scales) of a float64 matrix of float32 numbers.

    The quotient of two float32 numbers that is not a midpoint lies at least
    2^-29 of it away from one (w and mid * s are multiples of a common power of
    two, the latter with at most 29 bits), so float64 decides it."""
    W = np.asarray(W, dtype=np.float64)
    m, n = W.shape
    rb, cb = -(-m // block_rows), fp8_blocks(n)
    scales = np.ones((rb, cb), dtype=np.float32)
    for i in range(rb):
        for j in range(cb):
            top = np.max(np.abs(W[i * block_rows:(i + 1) * block_rows, j * FP8_BLOCK:(j + 1) * FP8_BLOCK]))
            if not np.isfinite(top):
                scales[i, j] = np.nan
            elif top > 0:
                scales[i, j] = max(np.float32(top / FP8_MAX), np.float32(2.0 ** -126))
    s = fp8_spread(scales, block_rows, m, n)
    with np.errstate(invalid="ignore"):
        codes = fp8_nearest_code(W / s)
    return np.where(np.isnan(s), 0, codes), scales


def fp8_dequantize(codes, scales, block_rows: int):
    codes = np.asarray(codes)
    return FP8_VALUES[codes] * fp8_spread(scales, block_rows, *codes.shape)


def fp8_error_bound(n: int, mags):
    """Bound on the error of products of codes widened to 16 bits, before the
    rounding to Y's type.  mags: sum of the terms' magnitudes.

    The matrix instructions round a block's running sum once for every eight
    columns (16 times a block, at most 2^-24 of the block's magnitudes each) and
    cut the eight terms and the sum 2^-24 below the largest (9 times 2^-24 of
    it, the largest terms adding up to the magnitudes at most); the product of
    the two scales and the last of the block's steps round once more.  That is
    27 times 2^-24 of each block's magnitudes, so of mags.  Adding the n / 128
    blocks rounds by 2^-24 of mags each, and at most 16 partial sums are then
    added.  In units of 2^-23: 14 + n / 256 + 8, and the rest of the 40 covers
    that the sums as rounded are a little larger than mags.  Results below
    float32's normal range round by 2^-150 each."""
    return (n / 256 + 40) * 2.0 ** -23 * mags + n * 2.0 ** -149


def fp8_stored_bound(n: int, mags, cut_mags):
    """A wider bound, that of the matrix instructions on 8-bit operands, which the
    products do not use: each instruction adds its products eight at a time and
    cuts each at 2^-13 of the largest of them as their exponents have it (codes
    below 2^-6 share its exponent): seven cuts of at most 2^-13 of the largest in
    eight, less than 2^-10 of cut_mags, the sum of the magnitudes with every
    non-zero code taken as at least 2^-6."""
    return fp8_error_bound(n, mags) + 2.0 ** -10 * cut_mags


def fp8_matmul(codes, scales, x_codes, x_scales):
    """X W^T, the sum of the terms' magnitudes, and that sum with non-zero codes
    of at least 2^-6 (float64; weights in blocks of 128 rows, X row by row)."""
    def parts(c, s, rows):
        v = FP8_VALUES[np.asarray(c)]
        f = fp8_spread(s, rows, *v.shape)
        a = np.abs(v)
        return v * f, a * np.abs(f), np.where(a > 0, np.maximum(a, 2.0 ** -6), 0.0) * np.abs(f)

    w, x = parts(codes, scales, FP8_BLOCK), parts(x_codes, x_scales, 1)
    return tuple(a @ b.T for a, b in zip(x, w))

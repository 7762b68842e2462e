"""Float64 reference of the microscaled (MXFP4) format and its products.

Elements are 4-bit e2m1 codes (bit 3 the sign, bits 0-2 the magnitude index
into MX_VALUES), every 32 consecutive columns of a row share one factor
2^(byte - 127) (byte 255: NaN).  Written from the format's definition: the
nearest code is found by comparing against every grid value.
"""
from __future__ import annotations

import numpy as np

MX_BLOCK = 32
MX_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MX_EMAX = 2                       # 6 = 1.5 * 2^2


def mx_blocks(n: int) -> int:
    return -(-n // MX_BLOCK)


def mx_block_byte(block) -> int:
    """Scale byte of one block of finite or non-finite float64 values."""
    top = float(np.max(np.abs(block))) if len(block) else 0.0
    if not np.isfinite(top):
        return 255
    if top == 0.0:
        return 127
    return max(int(np.frexp(top)[1]) - 1 - MX_EMAX, -127) + 127


def mx_nearest_code(v: float) -> int:
    """Code of the grid value nearest to v, ties to the even code; the code of
    6 for everything beyond."""
    d = np.abs(MX_VALUES - min(abs(v), 6.0))
    best = np.flatnonzero(d == d.min())
    code = int(best[0]) if len(best) == 1 else int([c for c in best if c % 2 == 0][0])
    return code | (8 if np.signbit(v) else 0)


def mx_quantize(W):
    """(codes m x n, bytes m x ceil(n/32)) of a float64 matrix."""
    W = np.asarray(W, dtype=np.float64)
    m, n = W.shape
    codes = np.zeros((m, n), dtype=np.int64)
    scale = np.zeros((m, mx_blocks(n)), dtype=np.int64)
    mids = (MX_VALUES[1:] + MX_VALUES[:-1]) / 2
    for b in range(mx_blocks(n)):
        lo, hi = b * MX_BLOCK, min(n, (b + 1) * MX_BLOCK)
        with np.errstate(invalid="ignore"):
            scale[:, b] = [mx_block_byte(row) for row in W[:, lo:hi]]
        ok = scale[:, b] != 255
        v = np.ldexp(W[ok, lo:hi], (127 - scale[ok, b])[:, None])
        a = np.abs(v)
        # Midpoint i lies between codes i and i + 1: it goes to the even one.
        c = np.zeros(a.shape, dtype=np.int64)
        for i, t in enumerate(mids):
            c += (a > t) | ((a == t) & ((i + 1) % 2 == 0))
        codes[ok, lo:hi] = c | np.where(np.signbit(v), 8, 0)
    return codes, scale


def mx_dequantize(codes, scale):
    """Float64 values of codes under their block factors."""
    codes = np.asarray(codes, dtype=np.int64)
    n = codes.shape[1]
    v = MX_VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    byte = np.repeat(np.asarray(scale, dtype=np.int64), MX_BLOCK, axis=1)[:, :n]
    return np.where(byte == 255, np.nan, np.ldexp(v, byte - 127))


def mx_matmul(codes, scale, X):
    """X What^T and the sum of the terms' magnitudes, float64."""
    W = mx_dequantize(codes, scale)
    X = np.asarray(X, dtype=np.float64)
    return X @ W.T, np.abs(X) @ np.abs(W).T


def mx_error_bound(n: int, mags, columns: int = 8, parts: int = 1):
    """Bound on the kernels' error before the rounding to Y's type.

    The matrix instructions add `columns` exact products at a time (8 of 16-bit
    X, 32 of microscaled X) to the running sum and round the result to nearest:
    an error of at most 2^-24 of a sum that is at most mags, n / columns times
    (`parts` = 2: every product as two, for float16 X in a workgroup that meets
    a scale byte outside 104 .. 135).  Before that the terms of a step are aligned to the largest
    and cut 2^-24 below its power of two: at most 2^-24 of it for each of eight
    terms and the sum before; the steps' largest terms add up to mags at most,
    so all cuts together take 9 * 2^-24 * parts of mags (the scaled
    instructions' cuts, far lower, as well).  At most 16 partial sums are then
    added, 2^-24 of mags each.  In units of 2^-23: n / (2 columns) parts, less
    than 20 for the cuts, 8 for the joins, and the rest of the 80 covers that
    the sums as rounded are a little larger than mags.  Steps whose results are
    subnormal round by at most 2^-150 each."""
    return (n * parts / (2 * columns) + 80) * 2.0 ** -23 * mags + n * 2.0 ** -149


def mx_matmul_bound(n: int, mags):
    """Tolerance for data whose roundings do not line up: fewer units than
    mx_error_bound's n / 16, which sums built for it reach."""
    return (n / 32 + 80) * 2.0 ** -23 * mags

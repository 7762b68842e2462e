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


def mx_matmul_bound(n: int, mags):
    """Bound on a float32 accumulation of n exact products in the kernels'
    order: chains of n/32 instruction results, at most 32 (128) terms joined
    inside an instruction and at most 32 partial sums joined behind it, each
    addition off by at most one unit 2^-23 of a partial sum <= mags."""
    return (n / 32 + 80) * 2.0 ** -23 * mags

"""Matrices in e4m3 with a scale per block of 128, and their product -- TEST
INFRASTRUCTURE.

Defined in include/archead.h: s = fp32(amax * fp32(1 / 448)), at least 2^-126 (0 for a
block of zeros); codes nearest to the exact quotient, ties to even.  Quotients
are taken in fp64: x has at most 24 significant bits and s 24, so a quotient
that is no tie lies at least 2^-50 of itself away from one, and fp64 tells.
Pins live in tests/test_oracle_fp8.py: every code, exact fractions at ties.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def decode(codes: np.ndarray) -> np.ndarray:
    """e4m3 codes (uint8) -> fp64: sign, 4 exponent bits (bias 7), 3 of mantissa; 0x7f and 0xff are NaN."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


_VALUES = decode(np.arange(127, dtype=np.uint8))
_MIDDLES = (_VALUES[1:] + _VALUES[:-1]) / 2


def encode(q: np.ndarray) -> np.ndarray:
    """The codes nearest to fp64 values, ties to the even code, 448 beyond it, NaN -> 0x7f (sign kept)."""
    a = np.abs(q)
    low, high = np.searchsorted(_MIDDLES, a, "left"), np.searchsorted(_MIDDLES, a, "right")
    code = np.where(low % 2 == 0, low, high)
    code = np.where(np.isnan(q), 127, code).astype(np.uint8)
    return code | (np.signbit(q).astype(np.uint8) << 7)


def scale_of(amax: np.ndarray) -> np.ndarray:
    """fp32 scales of blocks with these largest magnitudes (exact in fp32)."""
    a = np.asarray(amax, dtype=np.float32)
    s = np.maximum(a * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -126))
    return np.where(a > 0, s, np.float32(0))


def quantize(x: np.ndarray, block_rows: int = 1):
    """(codes uint8 rows x cols, scales fp32): scales [ceil(cols/128), rows] for
    block_rows = 1, else [ceil(rows/128), ceil(cols/128)].  x: finite fp32 values."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb, rb = -(-cols // BLOCK), -(-rows // block_rows)
    codes, s = np.zeros((rows, cols), dtype=np.uint8), np.zeros((rb, nb), dtype=np.float32)
    for i in range(rb):
        for b in range(nb):
            part = (slice(i * block_rows, (i + 1) * block_rows), slice(b * BLOCK, (b + 1) * BLOCK))
            s[i, b] = scale_of(np.abs(x[part]).max())
            if s[i, b] > 0:
                codes[part] = encode(x[part] / float(s[i, b]))
    return codes, (s.T.copy() if block_rows == 1 else s)


def matmul(a, sa, b, sb):
    """(out, bound) in fp64: the product and the sum of its terms' magnitudes."""
    A, B = decode(a), decode(b)
    K = A.shape[1]
    A = A * np.repeat(sa.astype(np.float64), BLOCK, axis=0)[:K].T
    B = B * np.repeat(np.repeat(sb.astype(np.float64), BLOCK, axis=0)[:B.shape[0]], BLOCK, axis=1)[:, :K]
    return A @ B.T, np.abs(A) @ np.abs(B).T

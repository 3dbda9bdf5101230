"""Rows in blocks of 4-bit codes, their definitions in 64 bits (numpy)."""
from __future__ import annotations

import numpy as np

MXFP4, NVFP4 = 0, 1
# experts, positions, K and N that moe_block_product takes with pairs of CTAs
PAIRS = [(1, 4000, 4096, 1000), (1, 2500, 512, 2560), (3, 2001, 1056, 4096), (1, 4000, 256, 8192), (1, 2100, 992, 4100),
         (4, 4096, 512, 2048), (2, 2400, 128, 8192), (7, 2691, 288, 8192), (3, 1400, 2048, 1000), (16, 4462, 4096, 2048)]
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
FINE = np.array([b * 2.0 ** -9 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 10) for b in range(127)])


def nearest(a, grid):
    """Place of the nearest of the grid's values, ties to the even place, the last one above it."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def size(fmt):
    return 16 if fmt == NVFP4 else 32


def row_scale(x):
    """The least power of two from max|row| / 2688 up, at least 2^-126; 0 for a row of zeros."""
    m, e = np.frexp(np.abs(x).max(1) / 2688)
    return np.where(m > 0, np.exp2(np.maximum(np.where(m == 0.5, e - 1, e), -126)), 0)


def scale_bytes(x, fmt, g=None):
    most = np.abs(x).reshape(x.shape[0], -1, size(fmt)).max(2)
    if fmt == MXFP4:
        return np.where(most > 0, np.maximum(np.frexp(most)[1] - 3, -127), -127) + 127
    g = g[:, None]
    return np.where(g > 0, nearest(most / np.where(g > 0, 6 * g, 1), FINE), 0)


def scale_values(bytes_, fmt):
    """Bytes to numbers; NaN for the NaN bytes."""
    b = bytes_.astype(np.int64)
    if fmt == MXFP4:
        return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return np.where(b == 127, np.nan, FINE[np.minimum(b, 126)])


def codes(x, s, g=None):
    """Codes of x with block scales s (numbers), the sign as it is, 0 where the scale is 0."""
    d = np.repeat(s if g is None else s * g[:, None], x.shape[1] // s.shape[1], 1)
    c = nearest(np.abs(x) / np.where(d > 0, d, 1), GRID) + 8 * np.signbit(x)
    return np.where(d > 0, c, 0).astype(np.uint8)


def pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    c = np.empty(q.shape[:-1] + (2 * q.shape[-1],), np.uint8)
    c[..., 0::2], c[..., 1::2] = q & 15, q >> 4
    return c


def values(q, s, fmt):
    """code times block scale of codes [..., K / 2] and scale bytes."""
    c = unpack(q)
    v = np.where(c > 7, -1, 1) * GRID[c & 7]
    return v * np.repeat(scale_values(s, fmt), size(fmt), -1)

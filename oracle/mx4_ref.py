"""Float64 reference of the cache in e2m1 codes with microscales -- TEST INFRASTRUCTURE.

Plain NumPy, written from the definitions: 32 values of a row share a power-of-two scale; a code is the
nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), its sign in bit 3.
"""
from __future__ import annotations

import numpy as np

SIZES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GROUP = 32
MIN_EXP = -126


def scale_exponent(x):
    """log2 of the smallest power of two s >= 2^-126 with |x| <= 7 s for the finite x."""
    a = np.abs(x[np.isfinite(x)])
    a = float(a.max()) if a.size else 0.0
    e = MIN_EXP
    while a > 7.0 * 2.0 ** e:
        e += 1
    return e


def encode(x):
    """Codes of float64 x (already divided by the scale; NaN gives some code)."""
    a = np.minimum(np.nan_to_num(np.abs(x), nan=0.0, posinf=6.0), 6.0)
    best = np.zeros(a.shape, np.int64)
    for c in range(1, 8):  # nearer than the best so far, or as near with an even code
        d, was = np.abs(a - SIZES[c]), np.abs(a - SIZES[best])
        best = np.where((d < was) | ((d == was) & (c % 2 == 0)), c, best)
    return best.astype(np.uint8) | np.where(np.signbit(x), 8, 0).astype(np.uint8)


def pack(codes):
    """[..., D] codes -> [..., D / 2] bytes, the first of two in the low bits."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    b = np.asarray(b, np.uint8)
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (2 * b.shape[-1],))


def quantise(row):
    """(bytes [D / 2], scale bytes [D / 32]) of a float64 row [D]."""
    codes, scales = np.zeros(row.size, np.uint8), np.zeros(row.size // GROUP, np.uint8)
    for j in range(scales.size):
        x = row[GROUP * j:GROUP * (j + 1)]
        e = scale_exponent(x)
        codes[GROUP * j:GROUP * (j + 1)] = encode(x / 2.0 ** e)
        scales[j] = 255 if np.isnan(x).any() else e + 127
    return pack(codes), scales


def values(codes, scales):
    """float64 values [..., D] of bytes [..., D / 2] and scale bytes [..., D / 32]."""
    c = unpack(codes)
    x = SIZES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return x * np.repeat(s, GROUP, -1)


def append(codes, scales, new, q_indptr, prefix_lens, tables):
    """Pools after the rows new [rows, Hkv, D] (float64) were written."""
    codes, scales = codes.copy(), scales.copy()
    hkv, bs = codes.shape[1], codes.shape[2]
    for b, p in enumerate(prefix_lens):
        for i in range(q_indptr[b + 1] - q_indptr[b]):
            blk, off = tables[b][(p + i) // bs], (p + i) % bs
            for g in range(hkv):
                codes[blk, g, off], scales[blk, g, off] = quantise(new[q_indptr[b] + i, g])
    return codes, scales


def compact(pool, src, indptr, starts, tables):
    """A pool [num_blocks, Hkv, bs, ...] after its tokens were moved together."""
    old, new = pool, pool.copy()
    bs = pool.shape[2]
    for b, start in enumerate(starts):
        for i in range(indptr[b + 1] - indptr[b]):
            s, d = src[indptr[b] + i], start + i
            new[tables[b][d // bs], :, d % bs] = old[tables[b][s // bs], :, s % bs]
    return new

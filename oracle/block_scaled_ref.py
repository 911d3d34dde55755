"""Float64 references of the block-scaled cache and of windowed attention -- TEST INFRASTRUCTURE.

Plain NumPy, written from the definitions: a page (the tokens of one block and kv head) is held as
e4m3 codes and one power-of-two scale; attention dequantises the tokens a query sees and takes the
textbook softmax over them.  Beside the outputs, attention() gives what an error bound needs.
"""
from __future__ import annotations

import math

import numpy as np

from .ref_numpy import E4M3, decode_storage

#: the finite, non-negative e4m3 values in order; their index is their code
_VALUES = decode_storage(np.arange(127, dtype=np.uint8), E4M3)
MIN_SCALE = 2.0 ** -126


def encode(x):
    """e4m3 codes of float64 x: the nearest value, ties to the even code, +-448 at most; NaN 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=1e300)), 448.0)
    hi = np.clip(np.searchsorted(_VALUES, a), 1, 126)
    lo = hi - 1
    up, down = _VALUES[hi] - a, a - _VALUES[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    code = code.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def decode(codes):
    return decode_storage(np.asarray(codes, np.uint8), E4M3)


def scale_of(x):
    """The smallest power of two >= 2^-126 with max |finite x| <= 448 times it."""
    a = np.abs(x[np.isfinite(x)])
    a = float(a.max()) if a.size else 0.0
    s = MIN_SCALE
    while a > 448.0 * s:
        s *= 2.0
    return s


def power_of_two_at_least(s):
    p = MIN_SCALE
    while p < s:
        p *= 2.0
    return p


def append(codes, scales, new, q_indptr, prefix_lens, tables):
    """codes uint8 [num_blocks, Hkv, bs, D], scales float32 [num_blocks, Hkv], new float64
    [rows, Hkv, D]: returns the codes and scales after the rows were written."""
    codes, scales = codes.copy(), scales.copy()
    hkv, bs = codes.shape[1], codes.shape[2]
    for b, p in enumerate(prefix_lens):
        rows = new[q_indptr[b]:q_indptr[b + 1]]
        n = len(rows)
        for lb in range(p // bs, (p + n + bs - 1) // bs if n else 0):
            blk = tables[b][lb]
            first, end = max(p - lb * bs, 0), min(p + n - lb * bs, bs)  # new offsets of the block
            for g in range(hkv):
                x = rows[lb * bs + first - p:lb * bs + end - p, g]
                s = scale_of(x)
                old = float(scales[blk, g])
                if first > 0:  # tokens that stay
                    s = max(s, power_of_two_at_least(old))
                    if s != old:
                        codes[blk, g, :first] = encode(decode(codes[blk, g, :first]) * (old / s))
                codes[blk, g, first:end] = encode(x / s)
                scales[blk, g] = s
    return codes, scales


def values(codes, scales):
    """float64 [num_blocks, Hkv, bs, D] of a pool: codes times a scale per block and head (an
    array) or per tensor (a number); float pools pass through with scales None."""
    if scales is None:
        return np.asarray(codes, np.float64)
    s = np.asarray(scales, np.float64)
    return decode(codes) * (s[:, :, None, None] if s.ndim else s)


def rows_of(vals, table, start, count):
    """[count, Hkv, D]: positions start .. of a request."""
    bs = vals.shape[2]
    t = start + np.arange(count)
    return vals[np.asarray(table, np.int64)[t // bs], :, t % bs]


def visible(pos, keys, window, sinks):
    """Whether a query at position pos sees keys (arrays, broadcast)."""
    return (keys <= pos) & ((window == 0) | (keys > pos - window) | (keys < sinks))


def attention(kv, vv, q, q_indptr, prefix_lens, tables, hq, sm_scale, window=0, sinks=0):
    """Rows q[q_indptr[b] + i] [rows, Hq, D] at positions prefix_lens[b] + i over the pools' values
    kv, vv.  Returns out, lse and, per (row, head): `mass` = sum p |v| [rows, Hq, D], `terms` =
    the largest sm_scale * sum |q| |k| of a seen key, `knorm` = the largest sm_scale * sum |k|,
    `seen` = the number of keys, `vmax` = the largest |v| of a seen key."""
    rows, d = q.shape[0], q.shape[2]
    grp = hq // kv.shape[1]
    bs = kv.shape[2]
    out, mass = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse = np.full((rows, hq), -np.inf)
    terms, knorm, vmax = np.zeros((rows, hq)), np.zeros((rows, hq)), np.zeros((rows, hq))
    seen = np.zeros((rows, hq))
    for b, p in enumerate(prefix_lens):
        for i in range(q_indptr[b + 1] - q_indptr[b]):
            pos, r = p + i, q_indptr[b] + i
            if pos < 0:
                continue
            t = np.arange(pos + 1)
            t = t[visible(pos, t, window, sinks)]
            blk, off = np.asarray(tables[b], np.int64)[t // bs], t % bs
            for h in range(hq):
                k, v = kv[blk, h // grp, off], vv[blk, h // grp, off]
                s = (k @ q[r, h]) * sm_scale
                e = np.exp(s - s.max())
                e /= e.sum()
                out[r, h], mass[r, h] = e @ v, e @ np.abs(v)
                lse[r, h] = s.max() + math.log(np.exp(s - s.max()).sum())
                terms[r, h] = abs(sm_scale) * (np.abs(k) @ np.abs(q[r, h])).max()
                knorm[r, h] = abs(sm_scale) * np.abs(k).sum(1).max()
                seen[r, h], vmax[r, h] = len(t), np.abs(v).max()
    return out, lse, {"mass": mass, "terms": terms, "knorm": knorm, "seen": seen, "vmax": vmax}

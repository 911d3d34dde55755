"""Helpers of the tests that are about a kernel form: a float64 attention that is quick enough for
some thousand rows, and the kernels that a call launched."""
from __future__ import annotations

import re

import numpy as np

from oracle.block_scaled_ref import visible


def attention(kv, vv, q, q_indptr, prefix_lens, tables, hq, sm_scale, window=0, sinks=0):
    """oracle.block_scaled_ref.attention, all rows of a request and kv head at once."""
    rows, d = q.shape[0], q.shape[2]
    hkv, bs = kv.shape[1], kv.shape[2]
    grp = hq // hkv
    out, mass = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse = np.full((rows, hq), -np.inf)
    terms, knorm, vmax, seen = (np.zeros((rows, hq)) for _ in range(4))
    for b, p in enumerate(prefix_lens):
        r0, r1 = q_indptr[b], q_indptr[b + 1]
        if r1 <= r0 or p < 0:
            continue
        pos = p + np.arange(r1 - r0)[:, None]
        t = np.arange(p + r1 - r0)[None]
        see = visible(pos, t, window, sinks)
        some = see.any(0)
        t, see = t[0, some], see[:, None, some]           # [rows, 1, keys]
        blk, off = np.asarray(tables[b], np.int64)[t // bs], t % bs
        for g in range(hkv):
            k, v = kv[blk, g, off], vv[blk, g, off]
            heads = slice(g * grp, (g + 1) * grp)
            x = q[r0:r1, heads]
            s = np.where(see, (x @ k.T) * sm_scale, -np.inf)
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(-1, keepdims=True)
            e /= total
            out[r0:r1, heads], mass[r0:r1, heads] = e @ v, e @ np.abs(v)
            lse[r0:r1, heads] = (top + np.log(total))[..., 0]
            terms[r0:r1, heads] = abs(sm_scale) * np.where(see, np.abs(x) @ np.abs(k).T, 0).max(-1)
            knorm[r0:r1, heads] = abs(sm_scale) * np.where(see, np.abs(k).sum(1), 0).max(-1)
            vmax[r0:r1, heads] = np.where(see, np.abs(v).max(1), 0).max(-1)
            seen[r0:r1, heads] = see.sum(-1)
    return out, lse, {"mass": mass, "terms": terms, "knorm": knorm, "seen": seen, "vmax": vmax}


def launches(names):
    """{name: [template arguments as integers]} of the library's kernels among demangled names."""
    got = {}
    for full in names:
        m = re.search(r"(\w+_kernel)<([^<>]*)>", full)
        if m and "pkv::" in full:
            words = [w.strip().replace("(bool)", "").replace("(int)", "") for w in m.group(2).split(",")]
            args = [{"true": 1, "false": 0}.get(w, w) for w in words]
            got.setdefault(m.group(1), []).append([int(a) for a in args])
        elif "pkv::" in full:
            m = re.search(r"(\w+_kernel)\b", full)
            if m:
                got.setdefault(m.group(1), []).append([])
    return got


def profiled(call):
    """call()'s result, and launches() of the kernels that it ran (None where no tracer is to be had).
    call() may be made twice."""
    import torch
    from torch.profiler import ProfilerActivity, profile
    for _ in range(2):  # (a tracer's first use may come too late for its kernels)
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            result = call()
            torch.cuda.synchronize()
        names = [e.name for e in prof.events() if "pkv::" in e.name]
        if names:
            return result, launches(names)
    return result, None

"""Helpers of the tests of the microscaled cache: small paged cases, calls and references.

Attention outputs are held to the bound of scaled_testlib (scores exact up to fp32 sums, since a code has
two significant bits and a scale is a power of two; weights in f16), with one more term where asked for
(`flushed`): decode takes V's scales into the weights relative to a reference of at least 2^-7 of the
largest one, f16 from 2^-14 up, so that a token whose scale is 2^-20 of the largest, and whose values are
then at most 6 2^-20 of it, may add nothing: 2^-17 vmax for vmax > 3.5 scales.
"""
from __future__ import annotations

import numpy as np
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from oracle import mx4_ref as M
from tests.pkv_testlib import to_f64
from tests.scaled_testlib import TDT, ints


def indptr(rows):
    return [0] + [int(x) for x in np.cumsum(rows)]


class Mx4Case:
    """Pools of random codes and scale bytes, and the requests' tables (lens: tokens held)."""

    def __init__(self, act, hkv, d, bs, lens, seed, spread=(118, 124), spare=3, width=None):
        rng = np.random.default_rng(seed)
        self.act, self.hkv, self.d, self.bs, self.lens, self.rng = act, hkv, d, bs, list(lens), rng
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + spare
        perm = rng.permutation(nb).astype(np.int32)
        self.tables = np.full((len(lens), width or max(max(need), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        codes = lambda: torch.from_numpy(rng.integers(0, 256, (nb, hkv, bs, d // 2)).astype(np.uint8))  # noqa: E731
        scales = lambda: torch.from_numpy(rng.integers(spread[0], spread[1] + 1, (nb, hkv, bs, d // 32)).astype(np.uint8))  # noqa: E731
        self.k, self.v, self.ks, self.vs = codes(), codes(), scales(), scales()

    def rows(self, n, heads, scale=1.0):
        x = torch.from_numpy((self.rng.standard_normal((n, heads, self.d)) * scale).astype(np.float32))
        return x.to(TDT[self.act])

    def cuda(self):
        for name in ("k", "v", "ks", "vs"):
            setattr(self, name, getattr(self, name).cuda())
        self.bt = torch.from_numpy(self.tables).cuda()
        return self

    def values(self):
        return [M.values(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((self.k, self.ks), (self.v, self.vs))]


def run_decode(c, q, hq, lens, window=0, sinks=0, splits=0, most=None):
    most = max(lens) if most is None else most
    out = torch.full((len(lens), hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((len(lens), hq), float("nan"), device="cuda")
    n = pkv.decode_mx4_workspace_bytes(c.k, len(lens), hq, most, window, sinks, splits)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    pkv.paged_decode_attn_mx4(c.k, c.v, c.ks, c.vs, q, out, c.bt, ints(lens), 1 / c.d ** 0.5, most, window=window,
                              sink_tokens=sinks, num_splits=splits, lse_out=lse, workspace=ws)
    return out, lse


def decode_ref(c, q, hq, lens, window=0, sinks=0):
    return R.attention(*c.values(), to_f64(q), range(len(lens) + 1), [n - 1 for n in lens], c.tables, hq, 1 / c.d ** 0.5,
                       window, sinks)


def run_extend(c, q, hq, rows, prefix, window=0, sinks=0, work=True):
    out = torch.full((q.shape[0], hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((q.shape[0], hq), float("nan"), device="cuda")
    ws = torch.full((pkv.extend_mx4_workspace_bytes(c.k),), 0xFF, dtype=torch.uint8, device="cuda") if work else None
    pkv.paged_extend_attn_mx4(c.k, c.v, c.ks, c.vs, q, out, ints(indptr(rows)), ints(prefix), c.bt, 1 / c.d ** 0.5,
                              max(rows), max(p + n for p, n in zip(prefix, rows)), window=window, sink_tokens=sinks,
                              lse_out=lse, workspace=ws)
    return out, lse


def extend_ref(c, q, hq, rows, prefix, window=0, sinks=0):
    return R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / c.d ** 0.5, window, sinks)

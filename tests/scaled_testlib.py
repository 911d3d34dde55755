"""Helpers of the block-scaled and window tests: small paged cases with every kind of cache, and
the bound that attention outputs are held to.

The bound of one output, from the kernels' arithmetic (u16 = half a step of f16, 2^-11; fp32 steps
2^-23):
  * scores: products of two values of at most 11 bits are exact in fp32; their sum over D terms is
    off by at most D 2^-23 sum |q k|; scaling, max and exp2 add 2^-21 relative; bf16 queries taken
    as f16 are off by at most 2^-25 each.  E = D 2^-23 terms + 2^-25 knorm + 2^-21 (1 + |lse|) is
    then the relative error of a weight, and the error of the lse with its own rounding;
  * weights as f16: u16 relative, or 2^-25 where a weight is subnormal (the largest weight is at
    least 1 when they are rounded);
  * V as f16: 2^-25 where it is subnormal; sums over n keys in fp32: n 2^-23;
  * the output's own rounding: half its last place.
So |out - ref| <= half_ulp + mass (u16 + 2 E + n 2^-23) + (n vmax + 1) 2^-25.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import block_scaled_ref as R
from tests.pkv_testlib import BF16, E4M3, F16, half_ulp, to_f64

TDT = {F16: torch.float16, BF16: torch.bfloat16}
SCALED = "scaled"


class Case:
    """A pool, its scales and the requests' tables.  cache: F16, BF16, E4M3 (one scale per tensor)
    or SCALED; lens: tokens per request (all held)."""

    def __init__(self, cache, act, hkv, d, bs, lens, seed, spread=(-8, -4), spare=3, width=None):
        rng = np.random.default_rng(seed)
        self.cache, self.act, self.hkv, self.d, self.bs, self.lens = cache, act, hkv, d, bs, list(lens)
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + spare
        perm = rng.permutation(nb).astype(np.int32)
        width = width or max(max(need), 1)
        self.tables = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        shape = (nb, hkv, bs, d)
        self.k_scale = self.v_scale = 1.0
        self.ks = self.vs = None
        pools = []
        for _ in range(2):
            x = rng.standard_normal(shape)
            if cache in (F16, BF16):
                pools.append(torch.from_numpy(x.astype(np.float32)).to(TDT[cache]))
            else:
                pools.append(torch.from_numpy(R.encode(x * 60)))
        self.k, self.v = pools
        if cache == E4M3:
            self.k_scale, self.v_scale = float(np.float32(0.017)), float(np.float32(0.013))
        if cache == SCALED:
            draw = lambda: np.exp2(rng.integers(spread[0], spread[1] + 1, (nb, hkv))).astype(np.float32)  # noqa: E731
            self.ks, self.vs = torch.from_numpy(draw()), torch.from_numpy(draw())
        self.rng = rng

    def rows(self, n, heads, scale=1.0):
        x = torch.from_numpy((self.rng.standard_normal((n, heads, self.d)) * scale).astype(np.float32))
        return x.to(TDT[self.act])

    def cuda(self):
        for name in ("k", "v", "ks", "vs"):
            t = getattr(self, name)
            if t is not None:
                setattr(self, name, t.cuda())
        self.bt = torch.from_numpy(self.tables).cuda()
        return self

    def values(self):
        """Float64 values of the K and V pools."""
        got = []
        for t, s, one in ((self.k, self.ks, self.k_scale), (self.v, self.vs, self.v_scale)):
            if self.cache in (F16, BF16):
                got.append(to_f64(t))
            else:
                codes = t.cpu().view(torch.uint8).numpy()
                got.append(R.values(codes, one if s is None else s.cpu().numpy()))
        return got


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def check_attention(out, lse, ref, act, d, what=""):
    want, want_lse, x = ref
    got, got_lse = to_f64(out), lse.cpu().double().numpy()
    none = np.isneginf(want_lse)
    assert np.all(np.isneginf(got_lse) == none) and np.all(got[none] == 0), what
    e = d * 2.0 ** -23 * x["terms"] + 2.0 ** -25 * x["knorm"] + 2.0 ** -21 * (1 + np.abs(np.where(none, 0, want_lse)))
    n = x["seen"][..., None]
    tol = half_ulp(want, act) + x["mass"] * (2.0 ** -11 + 2 * e[..., None] + n * 2.0 ** -23) + \
        (n * x["vmax"][..., None] + 1) * 2.0 ** -25
    off = np.abs(got - want)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    assert np.all(off <= tol), f"{what}: off {np.max(off)}, {np.max(off / np.maximum(tol, 1e-300))} of its bound"
    off = np.abs(np.where(none, 0, got_lse) - np.where(none, 0, want_lse))
    assert np.all(off <= e + n[..., 0] * 2.0 ** -23), f"{what}: lse off {np.max(off)}"

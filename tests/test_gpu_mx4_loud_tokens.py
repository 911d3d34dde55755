"""GPU checks of decode over microscaled codes whose V scales lie far apart: an output is held to the size of
the values that its weights give, however large a token's values are whose weight is next to nothing.

The bound of one output, from the kernel's arithmetic (w a token's weight, s its scale for the output's 32
dims, |v| <= 6 s; L2 norms are not used, every term is a worst case):
  * scores, as in scaled_testlib but token by token: e = D 2^-23 terms + 2^-25 knorm + 2^-21 (1 + |lse|) is
    the relative error of a weight, twice that with the sum's;
  * weights times scales in f16: 2^-11 relative, once for the weight and (slow path) once for the product;
    where they are subnormal less than themselves, and less than 2^-25 in units of the reference, which is at
    most 2^8 scales of a token that shares one with others, and 2^-4 of the largest weight: min(w, 2^-21) s,
    twice (the weight's own step, and the product's);
  * tokens that share no reference (tiles of 16): 2^-25 of twice the largest w s of the tile, for each token;
  * fp32 sums over n tokens: n 2^-23; the output's own rounding: half its last place.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from oracle import mx4_ref as M
from tests import paths_testlib as P
from tests.mx4_testlib import Mx4Case, run_decode
from tests.pkv_testlib import BF16, F16, half_ulp, to_f64

pytestmark = pytest.mark.gpu


def check(c, q, hq, lens, out, lse, window=0, sinks=0, what=""):
    kv, vv = c.values()
    scales = np.repeat(np.exp2(c.vs.cpu().numpy().astype(np.float64) - 127), 32, -1)
    got, got_lse, qv = to_f64(out), lse.cpu().double().numpy(), to_f64(q)
    sm, d, worst = 1 / c.d ** 0.5, c.d, 0.0
    for b, n in enumerate(lens):
        t = np.arange(n)
        t = t[R.visible(n - 1, t, window, sinks)]
        blk, off = c.tables[b].astype(np.int64)[t // c.bs], t % c.bs
        for h in range(hq):
            g = h // (hq // c.hkv)
            k, v, s = kv[blk, g, off], vv[blk, g, off], scales[blk, g, off]
            x = (k @ qv[b, h]) * sm
            w = np.exp(x - x.max())
            want_lse = x.max() + np.log(w.sum())
            w = (w / w.sum())[:, None]
            want = (w * v).sum(0)
            e = (d * 2.0 ** -23 * sm * (np.abs(k) @ np.abs(qv[b, h])) + 2.0 ** -25 * sm * np.abs(k).sum(1))[:, None] + \
                2.0 ** -21 * (1 + abs(want_lse))
            mass = np.abs(w * v).sum(0)
            both = (w[:, 0] * e[:, 0]).sum()
            tol = half_ulp(want, c.act) + (w * np.abs(v) * (2.0 ** -10 + e + both)).sum(0) + len(t) * 2.0 ** -23 * mass + \
                12 * (np.minimum(w, 2.0 ** -21) * s).sum(0) + 16 * 6 * 2.0 ** -24 * (w * s).sum(0)
            off_by = np.abs(got[b, h] - want)
            assert np.all(off_by <= tol), (what, b, h, np.max(off_by / tol), np.max(np.abs(want)))
            worst = max(worst, np.max(off_by / tol))
            assert abs(got_lse[b, h] - want_lse) <= both + len(t) * 2.0 ** -23, (what, b, h)
    assert pkv.get_device_error() == 0
    return worst


def loud_case(act, hq, hkv, d, bs, lens, seed, loud, up, some_groups=False, low=(112, 116)):
    """Requests whose tokens `loud(n)` have V scales 2^up above the others', and keys that the even heads' queries
    shun (weights of about 2^-70) and the odd ones' pick."""
    c = Mx4Case(act, hkv, d, bs, lens, seed=seed, spread=low)
    c.ks[:] = 124
    base = c.rng.standard_normal((hkv, d))
    q = base.repeat(hq // hkv, 0)[None] * np.where(np.arange(hq) % 2, -1, 1)[None, :, None]
    q = q + 0.1 * c.rng.standard_normal((len(lens), hq, d))
    shun = M.pack(np.where(base > 0, 15, 7).astype(np.uint8))        # -6 sign(base)
    for b, n in enumerate(lens):
        for t in loud(n):
            if 0 <= t < n:
                at = (int(c.tables[b, t // bs]), slice(None), t % bs)
                c.k[at], c.ks[at] = torch.from_numpy(shun), 127
                groups = np.flatnonzero(c.rng.integers(0, 2, d // 32)) if some_groups else np.arange(d // 32)
                for g in groups:
                    c.vs[at + (int(g),)] += up
    return c.cuda(), torch.from_numpy(q.astype(np.float32)).to({F16: torch.float16, BF16: torch.bfloat16}[act]).cuda()


LOUD = {
    "first": lambda n: [3],
    "last": lambda n: [n - 2],
    "middle": lambda n: [n // 2, n // 2 + 1],
    "first tiles": lambda n: range(0, min(128, n - 40)),
    "last tiles": lambda n: range(max(n - 150, 40), n),
    "here and there": lambda n: range(5, n, 37),
}


@pytest.mark.parametrize("where", LOUD, ids=lambda w: w.replace(" ", "-"))
@pytest.mark.parametrize("act,hq,hkv,d,bs,up", [(BF16, 4, 2, 128, 16, u) for u in (9, 14, 26, 60)] +
                         [(F16, 16, 1, 64, 32, u) for u in (11, 16)])  # (odd heads' outputs are loud: f16's range)
def test_a_loud_token_without_weight(where, act, hq, hkv, d, bs, up):
    lens = [700, 333, 64, 41]
    c, q = loud_case(act, hq, hkv, d, bs, lens, up, LOUD[where], up, low=(112, 116) if act == BF16 else (108, 112))
    for splits in (0, 1, 3):
        out, lse = run_decode(c, q, hq, lens, splits=splits)
        check(c, q, hq, lens, out, lse, what=f"{where} {up} {splits}")


@pytest.mark.parametrize("where", ["first", "middle", "here and there"], ids=lambda w: w.replace(" ", "-"))
@pytest.mark.parametrize("act,d,window,sinks", [(BF16, 128, 130, 20), (BF16, 64, 300, 0), (F16, 128, 500, 5)])
def test_in_a_window(where, act, d, window, sinks):
    lens = [650, 400, 90]
    for up in (13, 16):
        c, q = loud_case(act, 8, 1, d, 16, lens, window, LOUD[where], up, some_groups=True, low=(108, 112))
        for splits in (0, 1):
            out, lse = run_decode(c, q, 8, lens, window, sinks, splits)
            check(c, q, 8, lens, out, lse, window, sinks, f"{where} {up} {splits}")


@pytest.mark.parametrize("d,window", [(128, 0), (64, 0), (128, 40)])
def test_many_short_requests(d, window):
    # CTAs of two warps
    lens = [int(n) for n in np.random.default_rng(d).integers(20, 90, 330)]
    c, q = loud_case(BF16, 4, 2, d, 16, lens, d, LOUD["here and there"], 21, some_groups=True)
    (out, lse), ran = P.profiled(lambda: run_decode(c, q, 4, lens, window))
    check(c, q, 4, lens, out, lse, window)
    assert ran is None or "decode_kernel" in ran


def test_scales_of_every_size_at_once():
    # every token's scale anywhere in 2^-60 .. 2^39, its weight too; and rows of zeros (scale byte 1) among them
    lens = [500, 130, 33, 1]
    for seed in range(3):
        c = Mx4Case(BF16, 1, 128, 16, lens, seed=seed)
        c.vs = torch.from_numpy(c.rng.integers(67, 167, c.vs.shape).astype(np.uint8))
        c.ks = torch.from_numpy(c.rng.integers(118, 127, c.ks.shape).astype(np.uint8))
        zero = torch.from_numpy(c.rng.integers(0, 4, c.vs.shape) == 0)
        c.vs[zero] = 1
        c.v[zero.repeat_interleave(16, -1)] = 0
        c.cuda()
        q = c.rows(4, 8).cuda()
        for splits in (0, 1):
            out, lse = run_decode(c, q, 8, lens, splits=splits)
            check(c, q, 8, lens, out, lse, what=f"{seed} {splits}")


def test_rows_of_zeros_among_others_change_nothing():
    # a zero group has the smallest scale; with any other one its codes give the same
    lens = [600, 77]
    c = Mx4Case(BF16, 2, 128, 16, lens, seed=11)
    zero = torch.from_numpy(c.rng.integers(0, 6, c.vs.shape) == 0)
    zero[int(c.tables[0, 2])] = True
    c.v[zero.repeat_interleave(16, -1)] = 0
    c.cuda()
    q = c.rows(2, 8).cuda()
    for splits in (0, 1):
        want = run_decode(c, q, 8, lens, splits=splits)
        kept = c.vs.clone()
        c.vs[zero.cuda()] = 1
        got = run_decode(c, q, 8, lens, splits=splits)
        check(c, q, 8, lens, *got)
        c.vs = kept
        assert all(np.max(np.abs(to_f64(g) - to_f64(w))) <= 2.0 ** -8 * np.max(np.abs(to_f64(w))) for g, w in zip(got, want))

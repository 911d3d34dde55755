"""GPU checks of the microscaled 4-bit cache: writing (bit for bit against the float64 reference),
reading back, decode and extend over it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from oracle import mx4_ref as M
from tests import paths_testlib as P
from tests.mx4_testlib import Mx4Case, decode_ref, extend_ref, indptr, run_decode, run_extend
from tests.pkv_testlib import BF16, F16, to_f64
from tests.scaled_testlib import TDT, check_attention, ints

pytestmark = pytest.mark.gpu


def run_append(c, kn, vn, rows, prefix, most=None):
    """Append on the GPU and by the reference; the whole pools are compared."""
    ip = indptr(rows)
    want = [M.append(codes.cpu().numpy(), scales.cpu().numpy(), to_f64(new), ip, prefix, c.tables)
            for codes, scales, new in ((c.k, c.ks, kn), (c.v, c.vs, vn))]
    pkv.kv_append_mx4(c.k, c.v, c.ks, c.vs, kn.cuda(), vn.cuda(), ints(ip), ints(prefix), c.bt,
                      max(rows) if most is None else most)
    torch.cuda.synchronize()
    for codes, scales, (wc, ws) in ((c.k, c.ks, want[0]), (c.v, c.vs, want[1])):
        np.testing.assert_array_equal(scales.cpu().numpy(), ws)
        got, keep = M.unpack(codes.cpu().numpy()), np.repeat(ws != 255, 32, -1)
        np.testing.assert_array_equal(np.where(keep, got, 0), np.where(keep, M.unpack(wc), 0))


APPENDS = [
    # hkv, prefix, rows
    (2, [0], [1]),
    (1, [0, 15, 16, 17, 31, 33], [1, 1, 1, 1, 1, 1]),
    (3, [0, 5, 16, 40], [16, 11, 0, 70]),
    (8, [3, 100, 0], [1, 250, 33]),            # uneven: a unit's request is searched
    (2, [7] * 70, [1] * 69 + [90]),            # more than 32 requests, searched
    (1, [0, 0], [0, 5]),
]


@pytest.mark.parametrize("cfg", APPENDS, ids=lambda c: f"h{c[0]}-b{len(c[1])}-r{sum(c[2])}")
@pytest.mark.parametrize("d,bs,act", [(64, 16, F16), (64, 32, BF16), (128, 16, BF16), (128, 32, F16)])
def test_append(cfg, d, bs, act):
    hkv, prefix, rows = cfg
    c = Mx4Case(act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows) + d + bs).cuda()
    n = sum(rows)
    mag = torch.from_numpy(np.exp2(c.rng.integers(-9, 6, (n, hkv, 1))).astype(np.float32)).to(TDT[act])
    run_append(c, c.rows(n, hkv) * mag, c.rows(n, hkv) * mag.flip(0), rows, prefix)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("act", [F16, BF16])
def test_append_special_values(act):
    # zeros, the type's largest and smallest values, limits 7 2^k, ties, infinities and NaN
    d, bs = 64, 16
    big = 65504.0 if act == F16 else 3.3895313892515355e38
    tiny = 2.0 ** -24 if act == F16 else 2.0 ** -133
    nan, inf = float("nan"), float("inf")
    specials = [[0.0], [big, -1.0], [tiny], [7.0, 5.0, 2.5, 3.5], [7.0625], [0.875, 0.4375], [inf, 3.0], [-inf, nan, 1.0],
                [inf], [nan], [-0.0, tiny], [6.5, -6.75, 0.25, 0.75, 1.25, -1.75]]
    rows = [3] * len(specials)
    c = Mx4Case(act, 1, d, bs, [3 + n for n in rows], seed=9).cuda()
    kn = torch.zeros(sum(rows), 1, d)
    for i, v in enumerate(specials):
        for j, x in enumerate(v):
            kn[3 * i + j % 3, 0, 5 + 7 * j] = x
            kn[3 * i + 1, 0, j] = x
    kn = kn.to(TDT[act])
    run_append(c, kn, kn.flip(0).contiguous(), rows, [3] * len(rows))
    assert pkv.get_device_error() == 0


def test_append_every_bf16_value():
    # every finite bf16 value beside a fixed largest one of its row's groups
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[torch.isfinite(bits)]
    x = bits[: bits.numel() // 128 * 128].view(-1, 1, 128)
    c = Mx4Case(BF16, 1, 128, 16, [x.shape[0]], seed=1).cuda()
    run_append(c, x, x.flip(2).contiguous(), [x.shape[0]], [0])
    perm = torch.from_numpy(np.random.default_rng(0).permutation(x.numel()))
    run_append(c, x.flatten()[perm].view(x.shape), x, [x.shape[0]], [0])


def test_append_reports_and_skips():
    c = Mx4Case(F16, 2, 64, 16, [40, 40, 40], seed=6).cuda()
    kn, vn = c.rows(9, 2).cuda(), c.rows(9, 2).cuda()

    def refused(code, qi, prefix, bt, most):
        before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
        pkv.kv_append_mx4(c.k, c.v, c.ks, c.vs, kn, vn, ints(qi), ints(prefix), bt, most)
        assert pkv.get_device_error() == code
        return [bool(torch.equal(a, b)) for a, b in zip(before, (c.k, c.v, c.ks, c.vs))]

    assert all(refused(3, [0, 3, 3, 3], [46, 0, 0], c.bt, 3))           # past the table (48 tokens)
    assert all(refused(3, [0, 3, 3, 3], [-1, 0, 0], c.bt, 3))           # a negative prefix
    assert all(refused(3, [0, 10, 10, 10], [0, 0, 0], c.bt, 10))        # rows the call does not have
    assert all(refused(3, [0, 5, 3, 3], [46, 0, 0], c.bt, 9))           # a falling indptr
    bad = c.bt.clone()
    bad[0, 0], bad[1, 0] = -1, c.k.shape[0]
    assert all(refused(2, [0, 1, 2, 2], [0, 0, 0], bad, 1))             # blocks outside the pool
    want = M.append(c.k.cpu().numpy(), c.ks.cpu().numpy(), to_f64(kn), [0, 2, 2, 2], [0, 0, 0], c.tables)
    assert not all(refused(3, [0, 5, 5, 5], [0, 0, 0], c.bt, 2))        # rows beyond the hint
    np.testing.assert_array_equal(c.k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(c.ks.cpu().numpy(), want[1])


@pytest.mark.parametrize("act", [F16, BF16])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (3, 128, 32), (8, 128, 16)])
def test_gather(act, hkv, d, bs):
    starts, rows = [0, 7, 33, 2, 50], [1, 40, 0, 130, 17]
    c = Mx4Case(act, hkv, d, bs, [s + n for s, n in zip(starts, rows)], seed=hkv + d, spread=(95, 142)).cuda()
    n = sum(rows)
    ko, vo = (torch.full((n + 3, hkv, d), 7.0, dtype=TDT[act], device="cuda") for _ in range(2))
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko, vo, ints(indptr(rows)), ints(starts), c.bt)
    assert pkv.get_device_error() == 0
    for got, vals in zip((ko, vo), c.values()):
        want = np.concatenate([R.rows_of(vals, t, s, m) for t, s, m in zip(c.tables, starts, rows)])
        want = torch.from_numpy(want)
        want = (want.clamp(-65504, 65504) if act == F16 else want).to(TDT[act])
        assert torch.equal(got[:n].cpu(), want)
        assert bool((got[n:] == 7.0).all())  # rows of no request


def test_gather_reports_and_every_scale():
    c = Mx4Case(BF16, 1, 128, 16, [64], seed=8).cuda()
    c.ks.view(-1)[:256] = torch.arange(256, dtype=torch.uint8, device="cuda")
    c.vs.fill_(127)
    bt = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    c.tables = bt.cpu().numpy()
    ko, vo = (torch.full((64, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko, vo, ints([0, 64]), ints([0]), bt)
    want = torch.from_numpy(R.rows_of(c.values()[0], c.tables[0], 0, 64)).to(torch.bfloat16)
    assert torch.equal(ko.cpu().nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    assert pkv.get_device_error() == 0
    bad = torch.tensor([[0, -1], [c.k.shape[0], 1]], dtype=torch.int32, device="cuda")
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko[:6], vo[:6], ints([0, 4, 6]), ints([14, 4]), bad)
    assert pkv.get_device_error() == 1 and bool((ko[2:6] == 0).all()) and bool((vo[2:6] == 0).all())
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko[:6], vo[:6], ints([0, 1, 2]), ints([-1, 32]), bad)
    assert pkv.get_device_error() == 3 and bool((ko[:2] == 0).all())


DECODES = [
    # hq, hkv, d, bs, act, lens
    (4, 1, 64, 16, F16, [37, 60, 16, 1]),
    (8, 2, 128, 16, BF16, [1, 15, 17, 0, 100]),
    (24, 2, 128, 32, F16, [5, 200, 33]),
    (5, 1, 64, 32, BF16, [700, 31]),
    (8, 8, 128, 16, BF16, [2300]),
]


@pytest.mark.parametrize("cfg", DECODES, ids=lambda c: f"h{c[0]}x{c[1]}-d{c[2]}-bs{c[3]}-a{c[4]}")
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_decode(cfg, splits, window, sinks):
    hq, hkv, d, bs, act, lens = cfg
    c = Mx4Case(act, hkv, d, bs, lens, seed=sum(lens)).cuda()
    q = c.rows(len(lens), hq).cuda()
    out, lse = run_decode(c, q, hq, lens, window, sinks, splits)
    check_attention(out, lse, decode_ref(c, q, hq, lens, window, sinks), act, d, f"{cfg} {splits} {window}")
    assert pkv.get_device_error() == 0


MANY = [
    # batch, hq, hkv, d, bs, act, most: splits of one length, joined by a second launch or not at all
    (28, 8, 8, 64, 16, BF16, 1100),
    (80, 16, 8, 128, 32, F16, 1000),
    (40, 18, 2, 64, 16, F16, 1500),
    (160, 1, 1, 128, 16, BF16, 2100),
]


@pytest.mark.parametrize("cfg", MANY, ids=lambda c: f"b{c[0]}h{c[1]}x{c[2]}d{c[3]}n{c[6]}")
def test_decode_of_many_requests(cfg):
    batch, hq, hkv, d, bs, act, most = cfg
    rng = np.random.default_rng(batch)
    lens = [most, 0, 1, 16, most - 1] + list(rng.integers(0, most // 32, batch - 25) + 16 * rng.integers(0, 2, batch - 25))
    lens += list(16 * rng.integers(4, most // 16, 20) + rng.integers(-1, 2, 20))  # at and beside splits' ends
    lens = [int(n) for n in rng.permutation(lens)]
    c = Mx4Case(act, hkv, d, bs, lens, seed=batch).cuda()
    q = c.rows(batch, hq).cuda()
    out, lse = run_decode(c, q, hq, lens, most=most)
    ref = decode_ref(c, q, hq, lens)
    check_attention(out, lse, ref, act, d, f"{cfg}")
    assert pkv.get_device_error() == 0
    # a request past the hint is reported, the others are what they were
    short = sorted(lens)[-2] - 40
    again, lse = run_decode(c, q, hq, lens, most=short)
    kept = [i for i, n in enumerate(lens) if n <= short]
    ref = [r[kept] if isinstance(r, np.ndarray) else {k: v[kept] for k, v in r.items()} for r in ref]
    check_attention(again[kept], lse[kept], ref, act, d, f"{cfg} hint")
    assert pkv.get_device_error() == 3 and bool(torch.isfinite(again).all())


@pytest.mark.parametrize("act,hq,hkv,d,bs,longest,window,sinks", [
    (BF16, 4, 2, 128, 16, 2600, 0, 0), (F16, 32, 4, 64, 32, 3100, 0, 0),
    (BF16, 4, 4, 128, 16, 4800, 3600, 33), (F16, 24, 8, 64, 32, 6000, 5000, 0), (BF16, 80, 1, 64, 16, 4500, 3600, 20)])
def test_decode_in_splits_of_falling_length(act, hq, hkv, d, bs, longest, window, sinks):
    # most requests short, some at, before and behind the ends of the splits
    batch, rng = 80, np.random.default_rng(longest)
    seen = min(longest, window + sinks) if window else longest
    long = [longest, longest - 1, longest - 16, 16 * (seen // 32), 16 * (seen // 64) + 1] + \
        [16 * int(seen * x / 16) + y for x in (0.3, 0.714, 0.715) for y in (-1, 0, 1, 16)]
    lens = [int(n) for n in rng.permutation(long + [0, 1] + list(rng.integers(0, 90, batch - len(long) - 2)))]
    c = Mx4Case(act, hkv, d, bs, lens, seed=longest)
    for b, n in enumerate(lens):                                # what lies behind the last token
        if n % bs:
            c.ks[int(c.tables[b, n // bs]), :, n % bs:], c.vs[int(c.tables[b, n // bs]), :, n % bs:] = 255, 255
    c.cuda()
    q = c.rows(batch, hq).cuda()
    (out, lse), ran = P.profiled(lambda: run_decode(c, q, hq, lens, window, sinks))
    ref = P.attention(*c.values(), to_f64(q), range(batch + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5, window, sinks)
    check_attention(out, lse, ref, act, d)
    assert pkv.get_device_error() == 0 and (ran is None or len(ran["merge_kernel"]) == 1), ran


@pytest.mark.parametrize("batch,hq,hkv,d,bs,act,most", [(90, 16, 8, 128, 16, BF16, 130), (80, 8, 8, 64, 32, F16, 400),
                                                         (330, 36, 2, 64, 16, BF16, 70), (700, 2, 1, 128, 32, F16, 33)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (25, 2)])
def test_decode_of_many_short_requests(batch, hq, hkv, d, bs, act, most, window, sinks):
    lens = [int(n) for n in np.random.default_rng(batch).integers(0, most + 1, batch)]
    lens[3], lens[batch - 1] = most, 0
    c = Mx4Case(act, hkv, d, bs, lens, seed=batch).cuda()
    q = c.rows(batch, hq).cuda()
    out, lse = run_decode(c, q, hq, lens, window, sinks)
    check_attention(out, lse, decode_ref(c, q, hq, lens, window, sinks), act, d)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_decode_scales_of_any_size(splits):
    # K's scales 40 binary orders apart (few keys count); V's rising, falling, and 60 orders apart
    lens = [300, 64, 500, 129]
    c = Mx4Case(BF16, 2, 128, 16, lens, seed=3)
    c.ks = torch.from_numpy(c.rng.integers(84, 125, c.ks.shape).astype(np.uint8))
    c.vs = torch.from_numpy(c.rng.integers(60, 121, c.vs.shape).astype(np.uint8))
    for b, step in ((2, 1), (3, -1)):
        for i, blk in enumerate(c.tables[b, :-(-lens[b] // 16)]):
            c.vs[blk] = 100 + step * 2 * i
    c.cuda()
    q = c.rows(4, 8).cuda()
    out, lse = run_decode(c, q, 8, lens, splits=splits)
    ref = decode_ref(c, q, 8, lens)
    got, want, x = to_f64(out), ref[0], ref[2]
    # the bound of check_attention, and what tokens of small scales may add
    tol = 2.0 ** -8 * np.abs(want) + x["mass"] * 2.0 ** -10 + x["vmax"][..., None] * (2.0 ** -17 + x["seen"][..., None] * 2.0 ** -24)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    e = 128 * 2.0 ** -23 * x["terms"] + 2.0 ** -25 * x["knorm"] + 2.0 ** -21 * (1 + np.abs(ref[1])) + x["seen"] * 2.0 ** -23
    assert np.all(np.abs(lse.cpu().double().numpy() - ref[1]) <= e)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("d,act", [(64, BF16), (128, BF16)])
def test_decode_scales_from_one_end_of_their_range_to_the_other(splits, d, act):
    # V's scale bytes 1 .. 13 in the first tokens, then 241 .. 243 among them (and the other way round): their
    # difference, 15 more, passes 255
    lens = [300, 300, 40]
    c = Mx4Case(act, 1, d, 16, lens, seed=8)
    low = c.rng.integers(1, 14, c.vs.shape).astype(np.uint8)
    high = c.rng.integers(241, 244, c.vs.shape).astype(np.uint8)
    mixed = np.where(c.rng.integers(0, 3, c.vs.shape[:3] + (1,)) == 0, low, high)
    c.vs = torch.from_numpy(mixed)
    for i in range(10):
        c.vs[c.tables[0, i]] = torch.from_numpy(low[c.tables[0, i]])
    for i in range(10, 19):
        c.vs[c.tables[1, i]] = torch.from_numpy(low[c.tables[1, i]])
    c.cuda()
    q = c.rows(3, 4).cuda()
    out, lse = run_decode(c, q, 4, lens, splits=splits)
    ref = decode_ref(c, q, 4, lens)
    got, want, x = to_f64(out), ref[0], ref[2]
    # as above; a token's value is at most vmax, so that the flushed ones and f16's least steps count to it
    tol = 2.0 ** -8 * np.abs(want) + x["mass"] * 2.0 ** -10 + x["vmax"][..., None] * (2.0 ** -17 + x["seen"][..., None] * 2.0 ** -24)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    assert np.max(np.abs(want)) > 2.0 ** 110 and pkv.get_device_error() == 0


def test_decode_ignores_what_lies_past_the_end_and_keeps_nan():
    c = Mx4Case(BF16, 1, 128, 16, [21, 40], seed=3)
    blk = c.tables[0, 1]
    c.ks[blk, :, 5:], c.vs[blk, :, 5:] = 255, 255            # NaN scales behind the last token
    c.cuda()
    q = c.rows(2, 4).cuda()
    out, lse = run_decode(c, q, 4, [21, 40])
    check_attention(out, lse, decode_ref(c, q, 4, [21, 40]), BF16, 128)
    good = out.clone()
    c.vs[int(c.tables[1, 1]), 0, 3, 2] = 255                 # a NaN group of V: its dims alone
    out, _ = run_decode(c, q, 4, [21, 40])
    assert torch.equal(out[0], good[0]) and bool(torch.isnan(out[1, :, 64:96]).all())
    assert torch.equal(out[1, :, :64], good[1, :, :64]) and torch.equal(out[1, :, 96:], good[1, :, 96:])
    c.ks[int(c.tables[0, 0]), 0, 3, 1] = 255                 # of K: the whole request
    out, lse = run_decode(c, q, 4, [21, 40])
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert pkv.get_device_error() == 0


def test_decode_bad_blocks_read_zeros():
    c = Mx4Case(F16, 2, 64, 16, [48, 20], seed=5).cuda()
    q = c.rows(2, 4).cuda()
    zero = c.tables[0, 1]
    c.bt[0, 1] = c.k.shape[0] + 7
    out, lse = run_decode(c, q, 4, [48, 20])
    assert pkv.get_device_error() == 1
    c.k[int(zero)], c.v[int(zero)] = 0, 0
    check_attention(out, lse, decode_ref(c, q, 4, [48, 20]), F16, 64)
    c.bt[0, 1] = -1
    again, _ = run_decode(c, q, 4, [48, 20])
    assert pkv.get_device_error() == 1 and torch.equal(again, out)


EXTENDS = [
    # hq, hkv, d, bs, act, prefix, rows
    (4, 1, 64, 16, F16, [0, 37], [1, 50]),
    (8, 2, 128, 16, BF16, [200, 0, 3, 64], [33, 140, 0, 1]),
    (3, 1, 128, 32, BF16, [300], [260]),
    (8, 8, 64, 32, BF16, [129, 5], [40, 131]),
    (10, 2, 128, 16, F16, [77], [90]),
    (4, 1, 128, 16, BF16, [40, 3], [1100, 5]),
]


@pytest.mark.parametrize("cfg", EXTENDS, ids=lambda c: f"h{c[0]}x{c[1]}-d{c[2]}-bs{c[3]}-a{c[4]}-r{max(c[6])}")
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3), (150, 0)])
def test_extend(cfg, window, sinks):
    hq, hkv, d, bs, act, prefix, rows = cfg
    c = Mx4Case(act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
    q = c.rows(sum(rows), hq).cuda()
    ref = extend_ref(c, q, hq, rows, prefix, window, sinks)
    for work in (False, True):
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks, work)
        check_attention(out, lse, ref, act, d, f"{cfg} {window} {work}")
    assert pkv.get_device_error() == 0


# few rows over many keys, many short requests, requests of very different lengths
REGIMES = [([3], [2100], 4, 0, 0), ([70], [900], 4, 600, 130), ([530], [60], 16, 200, 4), ([5, 9, 2] * 20, [33] * 60, 2, 0, 0),
           ([1] * 9 + [900], [40] * 10, 4, 0, 0), ([16, 1, 30], [1500, 700, 0], 8, 0, 0), ([8], [2500], 8, 700, 9)]


@pytest.mark.parametrize("cfg", REGIMES, ids=lambda c: f"b{len(c[0])}-r{max(c[0])}-p{max(c[1])}-h{c[2]}-w{c[3]}")
@pytest.mark.parametrize("d,bs,act", [(64, 32, F16), (128, 16, BF16)])
def test_extend_regimes(cfg, d, bs, act):
    rows, prefix, hq, window, sinks = cfg
    c = Mx4Case(act, 1, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
    q = c.rows(sum(rows), hq).cuda()
    ref = extend_ref(c, q, hq, rows, prefix, window, sinks)
    for work in (False, True):
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks, work)
        check_attention(out, lse, ref, act, d, f"{cfg} {work}")
    assert pkv.get_device_error() == 0


def test_extend_reports():
    c = Mx4Case(BF16, 1, 64, 16, [40, 40], seed=5).cuda()
    q = c.rows(10, 2).cuda()
    out = torch.full((10, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(pkv.extend_mx4_workspace_bytes(c.k), dtype=torch.uint8, device="cuda")
    call = lambda qi, pl, most: pkv.paged_extend_attn_mx4(c.k, c.v, c.ks, c.vs, q, out, ints(qi), ints(pl), c.bt, 0.1,  # noqa: E731
                                                          most, 48, workspace=ws)
    call([0, 5, 12], [0, 0], 7)          # rows that the call does not have: not computed
    assert pkv.get_device_error() == 3 and bool((out[5:] == 3.0).all()) and bool((out[:5] != 3.0).any())
    call([0, 5, 10], [0, 46], 5)         # past the table
    assert pkv.get_device_error() == 3
    c.bt[0, 0] = -5
    call([0, 5, 10], [20, 0], 5)
    assert pkv.get_device_error() == 1

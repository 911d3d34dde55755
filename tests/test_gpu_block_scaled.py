"""GPU checks of the cache with a scale per block and kv head: writing (bit for bit against the
float64 reference), reading back, decode and extend over it, and a run of them together."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from tests.pkv_testlib import BF16, E4M3, F16, to_f64
from tests.scaled_testlib import SCALED, TDT, Case, check_attention, ints

pytestmark = pytest.mark.gpu


def indptr(rows):
    return [0] + list(np.cumsum(rows))


def codes_of(t):
    c = t.cpu().view(torch.uint8).numpy().copy()
    c[(c & 0x7F) == 0x7F] = 0x7F  # NaN has no sign here
    return c


def run_append(c, kn, vn, rows, prefix, most=None):
    """Append on the GPU and by the reference; returns nothing, compares codes and scales of the
    whole pools (so everything that must be left alone is)."""
    ip = indptr(rows)
    want = []
    for codes, scales, new in ((c.k, c.ks, kn), (c.v, c.vs, vn)):
        want.append(R.append(codes.cpu().numpy(), scales.cpu().numpy(), to_f64(new), ip, prefix, c.tables))
    pkv.kv_append_block_scaled(c.k, c.v, c.ks, c.vs, kn.cuda(), vn.cuda(), ints(ip), ints(prefix), c.bt,
                               max(rows) if most is None else most)
    torch.cuda.synchronize()
    for codes, scales, (wc, ws) in ((c.k, c.ks, want[0]), (c.v, c.vs, want[1])):
        np.testing.assert_array_equal(scales.cpu().numpy(), ws)
        wc = wc.copy()
        wc[(wc & 0x7F) == 0x7F] = 0x7F
        np.testing.assert_array_equal(codes_of(codes), wc)


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
    c = Case(SCALED, act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows) + d + bs).cuda()
    n = sum(rows)
    # magnitudes from token to token, so that scales grow, stay, and start afresh
    mag = torch.from_numpy(np.exp2(c.rng.integers(-9, 6, (n, hkv, 1))).astype(np.float32)).to(TDT[act])
    run_append(c, c.rows(n, hkv) * mag, c.rows(n, hkv) * mag.flip(0), rows, prefix)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("act", [F16, BF16])
def test_append_special_values(act):
    # zeros, the type's largest and smallest values, ties of 448 2^k, infinities and NaN
    d, bs = 64, 16
    big = 65504.0 if act == F16 else 3.3895313892515355e38
    tiny = 2.0 ** -24 if act == F16 else 2.0 ** -133
    nan, inf = float("nan"), float("inf")
    specials = [[0.0], [big, -1.0], [tiny], [448.0], [450.0], [0.875, 0.4375], [inf, 3.0], [-inf, nan, 1.0], [inf],
                [nan], [-0.0, tiny]]
    prefix, rows = [4] * len(specials) + [0] * len(specials), [3] * (2 * len(specials))
    c = Case(SCALED, act, 1, d, bs, [p + n for p, n in zip(prefix, rows)], seed=9, spread=(-30, 3)).cuda()
    kn = torch.zeros(sum(rows), 1, d)
    for i, v in enumerate(specials + specials):
        for j, x in enumerate(v):
            kn[3 * i + j % 3, 0, 5 + 7 * j] = x
    kn = kn.to(TDT[act])
    run_append(c, kn, kn.flip(0).contiguous(), rows, prefix)
    assert pkv.get_device_error() == 0


def test_append_old_scales_that_are_not_powers_of_two():
    c = Case(SCALED, BF16, 2, 64, 16, [9, 20], seed=4)
    c.ks.uniform_(0.001, 3.0)
    c.vs.uniform_(0.001, 3.0)
    c.cuda()
    run_append(c, c.rows(5, 2), c.rows(5, 2), [2, 3], [7, 17])


def test_append_token_by_token():
    # 40 decode steps of three requests: the scales grow inside blocks, new blocks start afresh
    c = Case(SCALED, BF16, 2, 128, 16, [45, 60, 41], seed=5).cuda()
    c.ks.fill_(float("nan"))  # what blocks hold before their first token does not count
    c.vs.fill_(123.0)
    at = [0, 16, 0]
    for step in range(40):
        x = c.rows(3, 2, 0.01 * 1.2 ** step)
        run_append(c, x, c.rows(3, 2), [1, 1, 1], at)
        at = [p + 1 for p in at]
    assert pkv.get_device_error() == 0


def test_append_reports_and_skips():
    c = Case(SCALED, F16, 2, 64, 16, [40, 40, 40], seed=6).cuda()
    kn, vn = c.rows(9, 2).cuda(), c.rows(9, 2).cuda()

    def refused(code, qi, prefix, bt, most):
        before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
        pkv.kv_append_block_scaled(c.k, c.v, c.ks, c.vs, kn, vn, ints(qi), ints(prefix), bt, most)
        assert pkv.get_device_error() == code
        return [bool(torch.equal(a, b)) for a, b in zip(before, (c.k, c.v, c.ks, c.vs))]

    assert all(refused(3, [0, 3, 3, 3], [46, 0, 0], c.bt, 3))           # past the table (48 tokens)
    assert all(refused(3, [0, 3, 3, 3], [-1, 0, 0], c.bt, 3))           # a negative prefix
    assert all(refused(3, [0, 10, 10, 10], [0, 0, 0], c.bt, 10))        # rows the call does not have
    assert all(refused(3, [0, 5, 3, 3], [46, 0, 0], c.bt, 9))           # a falling indptr
    bad = c.bt.clone()
    bad[0, 0], bad[1, 0] = -1, c.k.shape[0]
    assert all(refused(2, [0, 1, 2, 2], [0, 0, 0], bad, 1))             # blocks outside the pool
    # rows beyond the hint: those within it are written
    ip = [0, 5, 5, 5]
    want = R.append(c.k.cpu().numpy(), c.ks.cpu().numpy(), to_f64(kn), [0, 2, 2, 2], [0, 0, 0], c.tables)
    assert not all(refused(3, ip, [0, 0, 0], c.bt, 2))
    np.testing.assert_array_equal(codes_of(c.k), want[0])
    np.testing.assert_array_equal(c.ks.cpu().numpy(), want[1])


GATHERS = [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16), (SCALED, F16), (SCALED, BF16)]


@pytest.mark.parametrize("cache,act", GATHERS)
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (3, 128, 32), (8, 128, 16)])
def test_gather(cache, act, hkv, d, bs):
    starts, rows = [0, 7, 33, 2, 50], [1, 40, 0, 130, 17]
    c = Case(cache, act, hkv, d, bs, [s + n for s, n in zip(starts, rows)], seed=hkv + d, spread=(-20, 9)).cuda()
    n = sum(rows)
    ko, vo = (torch.full((n + 3, hkv, d), 7.0, dtype=TDT[act], device="cuda") for _ in range(2))
    pkv.kv_gather(c.k, c.v, ko, vo, ints(indptr(rows)), ints(starts), c.bt, c.k_scale, c.v_scale, c.ks, c.vs)
    assert pkv.get_device_error() == 0
    for got, vals in zip((ko, vo), c.values()):
        want = np.concatenate([R.rows_of(vals, t, s, m) for t, s, m in zip(c.tables, starts, rows)])
        if cache == E4M3:  # rounded to fp32, then to the output
            want = torch.from_numpy(want).float().to(TDT[act])
        else:  # exact in fp32; f16 keeps finite values inside its range
            want = torch.from_numpy(want)
            want = (want.clamp(-65504, 65504) if act == F16 else want).to(TDT[act])
        assert torch.equal(got[:n].cpu(), want)
        assert bool((got[n:] == 7.0).all())  # rows of no request


def test_gather_reports_and_special_codes():
    c = Case(SCALED, F16, 1, 64, 16, [32, 32], seed=8).cuda()
    c.k.view(-1)[:256] = torch.arange(256, dtype=torch.uint8, device="cuda")  # block 0: every code
    c.ks[0] = 2.0 ** 8
    bt = torch.tensor([[0, -1], [c.k.shape[0], 1]], dtype=torch.int32, device="cuda")
    ko, vo = (torch.full((6, 1, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pkv.kv_gather(c.k, c.v, ko, vo, ints([0, 4, 6]), ints([0, 31]), bt, k_scales=c.ks, v_scales=c.vs)
    assert pkv.get_device_error() == 3                        # position 32 of request 1: past its table
    want = (torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double() * 256).clamp(-65504, 65504).half()
    assert torch.equal(ko[:4].cpu().view(-1).nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    assert bool((ko[5] == 0).all()) and bool((ko[4] != 7.0).all())
    pkv.kv_gather(c.k, c.v, ko, vo, ints([0, 4, 6]), ints([14, 4]), bt, k_scales=c.ks, v_scales=c.vs)
    assert pkv.get_device_error() == 1                        # blocks outside the pool: zeros
    assert bool((ko[2:] == 0).all()) and bool((vo[2:] == 0).all())
    pkv.kv_gather(c.k, c.v, ko, vo, ints([0, 1, 2]), ints([-1, -5]), bt, k_scales=c.ks, v_scales=c.vs)
    assert pkv.get_device_error() == 3 and bool((ko[:2] == 0).all())


def run_decode(c, q, hq, lens, window=0, sinks=0, splits=0, most=None):
    most = max(lens) if most is None else most
    out = torch.full((len(lens), hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((len(lens), hq), float("nan"), device="cuda")
    n = pkv.decode_window_workspace_bytes(c.k, len(lens), hq, most, window, sinks, splits)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    pkv.paged_decode_attn_block_scaled(c.k, c.v, c.ks, c.vs, q, out, c.bt, ints(lens), 1 / c.d ** 0.5, most,
                                       window=window, sink_tokens=sinks, num_splits=splits, lse_out=lse, workspace=ws)
    return out, lse


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
    c = Case(SCALED, act, hkv, d, bs, lens, seed=sum(lens)).cuda()
    q = c.rows(len(lens), hq).cuda()
    out, lse = run_decode(c, q, hq, lens, window, sinks, splits)
    ref = R.attention(*c.values(), to_f64(q), range(len(lens) + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5,
                      window, sinks)
    check_attention(out, lse, ref, act, d, f"{cfg} {splits} {window}")
    assert pkv.get_device_error() == 0


MANY = [
    # batch, hq, hkv, d, bs, act, most: enough CTAs for splits of falling length
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
    c = Case(SCALED, act, hkv, d, bs, lens, seed=batch).cuda()
    q = c.rows(batch, hq).cuda()
    assert pkv.decode_window_workspace_bytes(c.k, batch, hq, most) > 0
    out, lse = run_decode(c, q, hq, lens, most=most)
    ref = R.attention(*c.values(), to_f64(q), range(batch + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5)
    check_attention(out, lse, ref, act, d, f"{cfg}")
    assert pkv.get_device_error() == 0
    # a request past the hint is reported, the others are what they were
    short = sorted(lens)[-2] - 40
    again, _ = run_decode(c, q, hq, lens, most=short)
    kept = [i for i, n in enumerate(lens) if n <= short]
    ref = [r[kept] if isinstance(r, np.ndarray) else {k: v[kept] for k, v in r.items()} for r in ref]
    check_attention(again[kept], _[kept], ref, act, d, f"{cfg} hint")
    assert pkv.get_device_error() == 3 and bool(torch.isfinite(again).all())


@pytest.mark.parametrize("batch,hq,hkv,d,bs,act,most", [(90, 16, 8, 128, 16, BF16, 130), (80, 8, 8, 64, 32, F16, 400),
                                                         (330, 36, 2, 64, 16, BF16, 70), (700, 2, 1, 128, 32, F16, 33)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (25, 2)])
def test_decode_of_many_short_requests(batch, hq, hkv, d, bs, act, most, window, sinks):
    # more CTAs than fit at once (CTAs of two warps)
    lens = [int(n) for n in np.random.default_rng(batch).integers(0, most + 1, batch)]
    lens[3], lens[batch - 1] = most, 0
    c = Case(SCALED, act, hkv, d, bs, lens, seed=batch).cuda()
    q = c.rows(batch, hq).cuda()
    out, lse = run_decode(c, q, hq, lens, window, sinks)
    ref = R.attention(*c.values(), to_f64(q), range(batch + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5, window,
                      sinks)
    check_attention(out, lse, ref, act, d)
    assert pkv.get_device_error() == 0


def test_decode_scales_of_any_size():
    # V scales 60 binary orders apart, and scales that are no powers of two
    c = Case(SCALED, BF16, 2, 128, 16, [300, 64], seed=3)
    c.vs = torch.from_numpy(np.exp2(c.rng.integers(-40, 20, c.vs.shape)).astype(np.float32))
    c.ks.uniform_(0.002, 0.03)
    c.cuda()
    q = c.rows(2, 8).cuda()
    out, lse = run_decode(c, q, 8, [300, 64])
    ref = R.attention(*c.values(), to_f64(q), [0, 1, 2], [299, 63], c.tables, 8, 1 / 128 ** 0.5)
    check_attention(out, lse, ref, BF16, 128)


def test_decode_ignores_what_lies_past_the_end():
    c = Case(SCALED, BF16, 1, 64, 16, [21], seed=3)
    blk = c.tables[0, 1]
    c.k[blk, :, 5:], c.v[blk, :, 5:] = 0x7F, 0xFF            # NaN codes behind the last token
    c.cuda()
    q = c.rows(1, 4).cuda()
    out, lse = run_decode(c, q, 4, [21])
    ref = R.attention(*c.values(), to_f64(q), [0, 1], [20], c.tables, 4, 1 / 8)
    check_attention(out, lse, ref, BF16, 64)


def run_extend(c, q, hq, rows, prefix, window=0, sinks=0, fill=0xFF):
    out = torch.full((q.shape[0], hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((q.shape[0], hq), float("nan"), device="cuda")
    ws = None
    if fill is not None:
        ws = torch.full((pkv.extend_block_scaled_workspace_bytes(c.k),), fill, dtype=torch.uint8, device="cuda")
    pkv.paged_extend_attn_block_scaled(c.k, c.v, c.ks, c.vs, q, out, ints(indptr(rows)), ints(prefix), c.bt,
                                       1 / c.d ** 0.5, max(rows), max(p + n for p, n in zip(prefix, rows)),
                                       window=window, sink_tokens=sinks, lse_out=lse, workspace=ws)
    return out, lse


EXTENDS = [
    # hq, hkv, d, bs, act, prefix, rows
    (4, 1, 64, 16, F16, [0, 37], [1, 50]),
    (8, 2, 128, 16, BF16, [200, 0, 3, 64], [33, 140, 0, 1]),
    (3, 1, 128, 32, BF16, [300], [260]),
    (8, 8, 64, 32, BF16, [129, 5], [40, 131]),
    (10, 2, 128, 16, F16, [77], [90]),
]


@pytest.mark.parametrize("cfg", EXTENDS, ids=lambda c: f"h{c[0]}x{c[1]}-d{c[2]}-bs{c[3]}-a{c[4]}")
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3), (150, 0)])
def test_extend(cfg, window, sinks):
    hq, hkv, d, bs, act, prefix, rows = cfg
    c = Case(SCALED, act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
    q = c.rows(sum(rows), hq).cuda()
    out, lse = run_extend(c, q, hq, rows, prefix, window, sinks)
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, window, sinks)
    check_attention(out, lse, ref, act, d, f"{cfg} {window}")
    assert pkv.get_device_error() == 0


# (rows, prefix, heads, window, sinks): many rows per request (pages widened into the workspace, or
# not without one), few rows over many keys (split over clusters of 2, 4 and 8), some of whose parts
# hold no key that a row sees
REGIMES = [([40, 530], [100, 3], 8, 0, 0), ([530], [60], 16, 200, 4), ([9, 0, 33], [700, 50, 300], 4, 0, 0),
           ([3], [2100], 4, 0, 0), ([70], [900], 4, 600, 130), ([200], [520], 2, 300, 0)]


@pytest.mark.parametrize("cfg", REGIMES, ids=lambda c: f"r{max(c[0])}-p{max(c[1])}-h{c[2]}-w{c[3]}")
@pytest.mark.parametrize("d,bs,act", [(64, 32, F16), (128, 16, BF16)])
def test_extend_regimes(cfg, d, bs, act):
    rows, prefix, hq, window, sinks = cfg
    c = Case(SCALED, act, 1, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
    q = c.rows(sum(rows), hq).cuda()
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, window, sinks)
    for fill in (0xFF, None):
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks, fill)
        check_attention(out, lse, ref, act, d, f"{cfg} {fill}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,bs,act", [(8, 2, 128, 16, BF16), (5, 1, 64, 32, F16), (2, 2, 64, 16, BF16),
                                             (12, 1, 128, 32, F16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_extend_of_few_rows(hq, hkv, d, bs, act, window, sinks):
    # requests whose rows fit one row tile, alone and many, over short and long prefixes
    for rows, prefix in (([1, 5, 0, 9], [300, 0, 17, 640]), ([10], [1500]), ([3] * 12, list(range(0, 480, 40)))):
        c = Case(SCALED, act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
        q = c.rows(sum(rows), hq).cuda()
        ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, window, sinks)
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks, None)
        check_attention(out, lse, ref, act, d, f"{rows} {window}")
    assert pkv.get_device_error() == 0


# requests of different lengths, few enough to fit the GPU at once: the long ones are split
UNEVEN = [([70, 3, 40, 0, 1], [900, 10, 300, 77, 1500]), ([1, 90], [2000, 0]), ([33] * 9, [1000] * 9),
          ([2, 100, 5] + [1] * 30, [800, 790, 0] + [50] * 30)]


@pytest.mark.parametrize("rows,prefix", UNEVEN, ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("d,bs,act,window,sinks", [(64, 32, F16, 0, 0), (128, 16, BF16, 0, 0), (128, 16, BF16, 850, 9)])
def test_extend_of_uneven_requests(rows, prefix, d, bs, act, window, sinks):
    c = Case(SCALED, act, 2, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
    q = c.rows(sum(rows), 8).cuda()
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, 8, 1 / d ** 0.5, window, sinks)
    out, lse = run_extend(c, q, 8, rows, prefix, window, sinks, None)
    check_attention(out, lse, ref, act, d)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("d,bs,act", [(64, 32, F16), (128, 16, BF16)])
def test_extend_of_more_items_than_sms(d, bs, act):
    # widened pages (the workspace given) and codes; rows from none to many, several items per SM
    rows, prefix, hq = [0, 1100, 1, 0, 70, 2, 900], [9, 30, 40, 0, 200, 64, 0], 8
    c = Case(SCALED, act, 8, d, bs, [p + n for p, n in zip(prefix, rows)], seed=12).cuda()
    q = c.rows(sum(rows), hq).cuda()
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5)
    for fill in (0xFF, None):
        out, lse = run_extend(c, q, hq, rows, prefix, fill=fill)
        check_attention(out, lse, ref, act, d, f"{fill}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("rows,prefix", [([16], [16]), ([20], [1500]), ([140], [0])])
def test_extend_scales_of_any_size(rows, prefix):
    # V scales that f16 does not hold, K scales far apart, and pages of zeros under the least scale
    c = Case(SCALED, BF16, 2, 128, 16, [rows[0] + prefix[0]], seed=rows[0])
    c.vs = torch.from_numpy(np.exp2(c.rng.integers(-20, 5, c.vs.shape)).astype(np.float32)) * 1.37
    c.ks = torch.from_numpy(np.exp2(c.rng.integers(-30, -4, c.ks.shape)).astype(np.float32))
    blk = c.tables[0, 0]
    c.k[blk], c.v[blk], c.ks[blk], c.vs[blk] = 0, 0, 2.0 ** -126, 2.0 ** -126
    c.cuda()
    q = c.rows(rows[0], 8).cuda()
    vals = c.values()
    vals[1] = to_f64(torch.from_numpy(vals[1]).float().half())  # V takes part as f16(code * scale)
    ref = R.attention(*vals, to_f64(q), [0, rows[0]], prefix, c.tables, 8, 1 / 128 ** 0.5)
    out, lse = run_extend(c, q, 8, rows, prefix, fill=None)
    check_attention(out, lse, ref, BF16, 128)


def test_extend_with_shared_blocks_and_dirty_tail():
    # two requests read the same prefix blocks; codes behind the last token are NaN
    c = Case(SCALED, BF16, 2, 128, 16, [96, 96], seed=12)
    c.tables[1, :4] = c.tables[0, :4]
    for b in range(2):
        blk = c.tables[b, 5]
        c.k[blk, :, 9:], c.v[blk, :, 9:] = 0x7F, 0x7F
    c.cuda()
    rows, prefix = [25, 25], [64, 64]
    q = c.rows(50, 8).cuda()
    out, lse = run_extend(c, q, 8, rows, prefix)
    ref = R.attention(*c.values(), to_f64(q), [0, 25, 50], prefix, c.tables, 8, 1 / 128 ** 0.5)
    check_attention(out, lse, ref, BF16, 128)
    again, _ = run_extend(c, q, 8, rows, prefix, fill=0)      # whatever the workspace held
    assert torch.equal(again, out)


def test_extend_f16_values_beyond_the_range_stay_finite():
    # the code of 65504 under its scale of 256 stands for 65536, more than f16 holds
    c = Case(SCALED, F16, 1, 64, 16, [16], seed=13)
    c.v.fill_(0x78)  # 256
    c.vs.fill_(256.0)
    c.cuda()
    q = c.rows(16, 1).cuda()
    out, _ = run_extend(c, q, 1, [16], [0])
    assert bool((out == 65504.0).all())
    out, _ = run_decode(c, q[:1], 1, [16])                    # decode holds 65536 in fp32; f16 rounds it to inf
    assert bool(torch.isinf(out).all())




def test_a_run_of_all_calls():
    # append a prompt -> extend over it -> decode steps (append, attend) -> read back, against the
    # reference after every call
    hq, hkv, d, bs, act = 8, 2, 128, 16, BF16
    prompts, steps = [50, 7, 0, 33], 20
    c = Case(SCALED, act, hkv, d, bs, [n + steps for n in prompts], seed=21).cuda()
    rows = prompts
    run_append(c, c.rows(sum(rows), hkv), c.rows(sum(rows), hkv), rows, [0] * 4)
    q = c.rows(sum(rows), hq).cuda()
    out, lse = run_extend(c, q, hq, rows, [0] * 4, 24, 4)
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), [0] * 4, c.tables, hq, 1 / d ** 0.5, 24, 4)
    check_attention(out, lse, ref, act, d, "prompt")
    at = list(prompts)
    for i in range(steps):
        run_append(c, c.rows(4, hkv, 1 + 0.2 * i), c.rows(4, hkv, 1 + 0.1 * i), [1] * 4, at)
        at = [n + 1 for n in at]
        q = c.rows(4, hq).cuda()
        out, lse = run_decode(c, q, hq, at, 24, 4, most=80)
        ref = R.attention(*c.values(), to_f64(q), range(5), [n - 1 for n in at], c.tables, hq, 1 / d ** 0.5, 24, 4)
        check_attention(out, lse, ref, act, d, f"step {i}")
    ko, vo = (torch.empty((sum(at), hkv, d), dtype=TDT[act], device="cuda") for _ in range(2))
    pkv.kv_gather(c.k, c.v, ko, vo, ints(indptr(at)), ints([0] * 4), c.bt, k_scales=c.ks, v_scales=c.vs)
    for got, vals in zip((ko, vo), c.values()):
        want = np.concatenate([R.rows_of(vals, t, 0, m) for t, m in zip(c.tables, at)])
        assert np.array_equal(to_f64(got), want)
    assert pkv.get_device_error() == 0


def test_a_step_in_a_cuda_graph_and_on_two_streams():
    hq, hkv, d, bs, act = 8, 2, 64, 16, BF16
    lens = [40, 300]

    class Server:
        def __init__(self):
            self.c = c = Case(SCALED, act, hkv, d, bs, [n + 16 for n in lens], seed=31).cuda()
            self.kn, self.vn, self.q = c.rows(2, hkv).cuda(), c.rows(2, hkv).cuda(), c.rows(2, hq).cuda()
            self.qi, self.at, self.n = ints([0, 1, 2]), ints(lens), ints([m + 1 for m in lens])
            self.out = torch.empty_like(self.q)
            need = pkv.decode_window_workspace_bytes(c.k, 2, hq, 512, 0, 0, 4)
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def step(self, stream=None):
            c = self.c
            pkv.kv_append_block_scaled(c.k, c.v, c.ks, c.vs, self.kn, self.vn, self.qi, self.at, c.bt, 1, stream=stream)
            pkv.paged_decode_attn_block_scaled(c.k, c.v, c.ks, c.vs, self.q, self.out, c.bt, self.n, 1 / d ** 0.5, 512,
                                               num_splits=4, workspace=self.ws, stream=stream)

        def advance(self):
            self.at += 1
            self.n += 1

    one, two, graphed = Server(), Server(), Server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            graphed.step()
    for _ in range(10):
        one.step()
        two.step(stream=side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one.out, two.out) and torch.equal(one.out, graphed.out)
        assert torch.equal(one.c.k, graphed.c.k) and torch.equal(one.c.vs, graphed.c.vs)
        for s in (one, two, graphed):
            s.advance()
        torch.cuda.synchronize()
    ref = R.attention(*one.c.values(), to_f64(one.q), [0, 1, 2], [n + 9 for n in lens], one.c.tables, hq, 1 / d ** 0.5)
    lse = torch.from_numpy(ref[1])  # not computed here
    check_attention(one.out, lse, ref, act, d)
    assert pkv.get_device_error() == 0


def test_pools_beyond_32_bit_offsets():
    # 2.3 GB of codes per pool: blocks at the far end, through every call
    hq, hkv, d, bs = 8, 8, 128, 32
    nb = 70000
    k, v = (torch.zeros((nb, hkv, bs, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, hkv), device="cuda") for _ in range(2))
    small = Case(SCALED, BF16, hkv, d, bs, [100], seed=41)
    kn, vn, q = small.rows(100, hkv).cuda(), small.rows(100, hkv).cuda(), small.rows(100, hq).cuda()
    bt = torch.tensor([[nb - 1, nb - 7, 66000, 69000]], dtype=torch.int32, device="cuda")
    pkv.kv_append_block_scaled(k, v, ks, vs, kn, vn, ints([0, 100]), ints([0]), bt, 100)
    ko, vo = torch.empty_like(kn), torch.empty_like(vn)
    pkv.kv_gather(k, v, ko, vo, ints([0, 100]), ints([0]), bt, k_scales=ks, v_scales=vs)
    # the same at the start of a small pool
    small.tables = np.arange(4, dtype=np.int32)[None]
    small.cuda()
    pkv.kv_append_block_scaled(small.k, small.v, small.ks, small.vs, kn, vn, ints([0, 100]), ints([0]), small.bt, 100)
    ko2, vo2 = torch.empty_like(kn), torch.empty_like(vn)
    pkv.kv_gather(small.k, small.v, ko2, vo2, ints([0, 100]), ints([0]), small.bt, k_scales=small.ks, v_scales=small.vs)
    assert torch.equal(ko, ko2) and torch.equal(vo, vo2)
    outs = []
    for kk, vv, s1, s2, t in ((k, v, ks, vs, bt), (small.k, small.v, small.ks, small.vs, small.bt)):
        out, o2 = torch.empty_like(q[:1]), torch.empty_like(q)
        ws = torch.empty(pkv.decode_window_workspace_bytes(kk, 1, hq, 100, 0, 0, 2), dtype=torch.uint8, device="cuda")
        pkv.paged_decode_attn_block_scaled(kk, vv, s1, s2, q[:1], out, t, ints([100]), 0.1, 100, num_splits=2, workspace=ws)
        ws = torch.empty(pkv.extend_block_scaled_workspace_bytes(kk), dtype=torch.uint8, device="cuda")
        pkv.paged_extend_attn_block_scaled(kk, vv, s1, s2, q, o2, ints([0, 100]), ints([0]), t, 0.1, 100, 100, workspace=ws)
        outs.append((out, o2))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert int(k[:60000].max()) == 0 and pkv.get_device_error() == 0

"""GPU checks of attention with a sliding window and sink tokens, for every kind of cache."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from tests.pkv_testlib import BF16, E4M3, F16, to_f64
from tests.scaled_testlib import TDT, Case, check_attention, ints

pytestmark = pytest.mark.gpu


def indptr(rows):
    return [0] + list(np.cumsum(rows))


def give_back(c, first_pos, window, sinks):
    """Table entries of blocks that no query from first_pos[b] on sees become ids outside the pool,
    and those blocks' contents NaN; so do hidden tokens of the blocks that stay."""
    nan = 0x7F if c.k.dtype == torch.uint8 else float("nan")
    for b, p in enumerate(first_pos):
        for lb in range(-(-c.lens[b] // c.bs)):
            t = lb * c.bs + np.arange(c.bs)
            hidden = (t >= sinks) & (t < p - window + 1)
            blk = int(c.tables[b, lb])
            for off in np.flatnonzero(hidden):
                c.k[blk, :, off], c.v[blk, :, off] = nan, nan
            if hidden.all():
                c.tables[b, lb] = -1 if lb % 2 else c.k.shape[0] + 5


def run_decode(c, q, hq, lens, window, sinks, splits=0, most=None):
    most = max(lens) if most is None else most
    out = torch.full((len(lens), hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((len(lens), hq), float("nan"), device="cuda")
    n = pkv.decode_window_workspace_bytes(c.k, len(lens), hq, most, window, sinks, splits)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    pkv.paged_decode_attn_window(c.k, c.v, q, out, c.bt, ints(lens), 1 / c.d ** 0.5, most, window, sinks,
                                 k_scale=c.k_scale, v_scale=c.v_scale, num_splits=splits, lse_out=lse, workspace=ws)
    return out, lse


DECODES = [
    # cache, act, hq, hkv, d, bs, lens
    (F16, F16, 4, 1, 64, 16, [37, 60, 16, 1, 0]),
    (BF16, BF16, 8, 2, 128, 16, [15, 17, 100, 301]),
    (E4M3, F16, 3, 3, 64, 32, [200, 33]),
    (E4M3, BF16, 24, 2, 128, 32, [640, 90]),
    (BF16, BF16, 5, 1, 64, 16, [1500]),
    (F16, F16, 16, 2, 128, 32, [130, 5]),
]
WINDOWS = [(1, 0), (1, 1), (16, 0), (17, 4), (33, 16), (64, 100), (100, 1), (5000, 7), (2**31 - 1, 2**31 - 1)]


@pytest.mark.parametrize("cfg", DECODES, ids=lambda c: f"c{c[0]}a{c[1]}h{c[2]}x{c[3]}d{c[4]}bs{c[5]}")
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_decode(cfg, window, sinks):
    cache, act, hq, hkv, d, bs, lens = cfg
    for splits in (0, 3):
        c = Case(cache, act, hkv, d, bs, lens, seed=sum(lens) + window % 997)
        q = c.rows(len(lens), hq).cuda()
        give_back(c, [n - 1 for n in lens], window, sinks)
        c.cuda()
        out, lse = run_decode(c, q, hq, lens, window, sinks, splits)
        assert pkv.get_device_error() == 0
        ref = R.attention(*c.values(), to_f64(q), range(len(lens) + 1), [n - 1 for n in lens], c.tables, hq,
                          1 / d ** 0.5, window, sinks)
        check_attention(out, lse, ref, act, d, f"{cfg} {window} {sinks} {splits}")


@pytest.mark.parametrize("cache,act,hq,hkv,d,window,sinks", [(BF16, BF16, 4, 2, 128, 1800, 20), (F16, F16, 2, 2, 64, 3600, 0),
                                                               (E4M3, F16, 2, 2, 128, 3590, 33)])
def test_decode_of_many_requests(cache, act, hq, hkv, d, window, sinks):
    # splits of falling length in the numbering without the hidden tokens: most requests short,
    # some as long as the window, some longer
    batch, rng = 80, np.random.default_rng(window)
    long = [window, window + 1, window + 17, window + sinks + 700, window - 16, 16 * (window // 32), 16 * (window // 64) + 1]
    lens = [int(n) for n in rng.permutation(long + list(rng.integers(0, 90, batch - len(long))))]
    c = Case(cache, act, hkv, d, 16, lens, seed=window)
    q = c.rows(batch, hq).cuda()
    give_back(c, [n - 1 for n in lens], window, sinks)
    c.cuda()
    assert pkv.decode_window_workspace_bytes(c.k, batch, hq, max(lens), window, sinks) > 0
    out, lse = run_decode(c, q, hq, lens, window, sinks)
    assert pkv.get_device_error() == 0
    ref = R.attention(*c.values(), to_f64(q), range(batch + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5, window,
                      sinks)
    check_attention(out, lse, ref, act, d)


@pytest.mark.parametrize("cache,act,hq,hkv,d,window,sinks", [(BF16, BF16, 16, 4, 128, 128, 4), (F16, F16, 4, 4, 64, 300, 0),
                                                               (E4M3, F16, 8, 4, 128, 64, 33), (E4M3, BF16, 4, 4, 64, 17, 1)])
def test_decode_of_many_requests_in_a_short_window(cache, act, hq, hkv, d, window, sinks):
    # more CTAs than fit at once (CTAs of two warps)
    batch = 170
    lens = [int(n) for n in np.random.default_rng(window).integers(0, 500, batch)]
    c = Case(cache, act, hkv, d, 32, lens, seed=window)
    q = c.rows(batch, hq).cuda()
    give_back(c, [n - 1 for n in lens], window, sinks)
    c.cuda()
    out, lse = run_decode(c, q, hq, lens, window, sinks)
    assert pkv.get_device_error() == 0
    ref = R.attention(*c.values(), to_f64(q), range(batch + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5, window,
                      sinks)
    check_attention(out, lse, ref, act, d)


def test_decode_of_a_whole_window_is_the_plain_decode():
    lens = [700, 33, 1]
    c = Case(BF16, BF16, 2, 128, 16, lens, seed=3).cuda()
    q = c.rows(3, 8).cuda()
    plain = torch.empty_like(q)
    ws = torch.empty(max(pkv.decode_workspace_bytes(c.k, 3, 8, 700), 1), dtype=torch.uint8, device="cuda")
    pkv.paged_decode_attn(c.k, c.v, q, plain, c.bt, ints(lens), 1 / 128 ** 0.5, 700, workspace=ws)
    for window, sinks in ((700, 0), (1000, 5), (1, 700)):
        out, _ = run_decode(c, q, 8, lens, window, sinks)
        if window >= 700:
            assert torch.equal(out, plain)
        else:  # every token is a sink: the same tokens, split elsewhere
            assert torch.allclose(out.float(), plain.float(), rtol=2.0 ** -7, atol=1e-3)


def test_decode_reports():
    c = Case(BF16, BF16, 2, 64, 16, [100, 100], seed=4).cuda()
    q = c.rows(2, 4).cuda()
    bad = c.bt.clone()
    c.bt = bad
    bad[0, 6], bad[1, 0] = -1, 10 ** 6                         # the current token's block, a sink's block
    out, _ = run_decode(c, q, 4, [100, 100], 8, 3)
    assert pkv.get_device_error() == 1 and bool(torch.isfinite(out).all())
    c.bt = torch.from_numpy(c.tables).cuda()
    for lens in ([113, 5], [-2, 5]):                           # past the table, negative
        out, _ = run_decode(c, q, 4, lens, 8, 3, most=120)
        assert pkv.get_device_error() == 3
    # a length beyond the hint, without a window to bound the work
    run_decode(c, q, 4, [100, 5], 2000, 0, splits=1, most=16)
    assert pkv.get_device_error() == 3


def run_extend(c, q, hq, rows, prefix, window, sinks, widen=False):
    out = torch.full((q.shape[0], hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((q.shape[0], hq), float("nan"), device="cuda")
    ws = torch.full((max(pkv.extend_widen_workspace_bytes(c.k), 1),), 0xFF, dtype=torch.uint8, device="cuda") if widen else None
    pkv.paged_extend_attn_window(c.k, c.v, q, out, ints(indptr(rows)), ints(prefix), c.bt, 1 / c.d ** 0.5,
                                 max(rows), max(p + n for p, n in zip(prefix, rows)), window, sinks,
                                 k_scale=c.k_scale, v_scale=c.v_scale, lse_out=lse, workspace=ws)
    return out, lse


EXTENDS = [
    # cache, act, hq, hkv, d, bs, prefix, rows
    (F16, F16, 4, 1, 64, 16, [0, 37], [1, 90]),
    (BF16, BF16, 8, 2, 128, 16, [400, 0, 3, 64], [33, 140, 0, 1]),
    (E4M3, F16, 3, 1, 64, 32, [300], [260]),
    (E4M3, BF16, 8, 8, 128, 32, [129, 5], [40, 150]),
    (BF16, BF16, 12, 1, 64, 16, [500, 17], [30, 70]),
    (F16, F16, 2, 2, 128, 32, [250], [300]),
    (E4M3, BF16, 16, 2, 64, 16, [33], [70]),
]


@pytest.mark.parametrize("cfg", EXTENDS, ids=lambda c: f"c{c[0]}a{c[1]}h{c[2]}x{c[3]}d{c[4]}bs{c[5]}")
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_extend(cfg, window, sinks):
    cache, act, hq, hkv, d, bs, prefix, rows = cfg
    for widen in (False, True) if cache != F16 else (False,):
        c = Case(cache, act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows) + window % 997)
        q = c.rows(sum(rows), hq).cuda()
        give_back(c, prefix, window, sinks)
        c.cuda()
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks, widen)
        assert pkv.get_device_error() == 0
        ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, window, sinks)
        check_attention(out, lse, ref, act, d, f"{cfg} {window} {sinks} {widen}")


def test_extend_over_many_tiles():
    # sinks over more than one key tile, a window of several, a gap between them, and several items
    prefix, rows = [1500], [400]
    c = Case(BF16, BF16, 1, 128, 16, [1900], seed=17)
    q = c.rows(400, 2).cuda()
    window, sinks = 700, 200
    give_back(c, prefix, window, sinks)
    c.cuda()
    out, lse = run_extend(c, q, 2, rows, prefix, window, sinks)
    ref = R.attention(*c.values(), to_f64(q), [0, 400], prefix, c.tables, 2, 1 / 128 ** 0.5, window, sinks)
    check_attention(out, lse, ref, BF16, 128)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("cache,act,d", [(BF16, BF16, 128), (E4M3, BF16, 64), (F16, F16, 128)])
def test_extend_of_more_items_than_sms(cache, act, d):
    # several items per SM, taken as they come: requests of one row beside requests of many, empty
    # requests, and pairs past a short request's rows in between
    rows = [0, 1, 330, 0, 0, 2, 700, 1, 64, 65, 0, 500, 3, 1, 129, 0]
    prefix = [9, 40, 0, 5, 0, 33, 100, 0, 70, 5, 1, 260, 0, 300, 16, 0]
    hq, hkv = 8, 8
    c = Case(cache, act, hkv, d, 16, [p + n for p, n in zip(prefix, rows)], seed=11).cuda()
    q = c.rows(sum(rows), hq).cuda()
    out, lse = run_extend(c, q, hq, rows, prefix, 150, 5)
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, 150, 5)
    check_attention(out, lse, ref, act, d)
    again, _ = run_extend(c, q, hq, rows, prefix, 150, 5)
    assert torch.equal(again, out)
    assert pkv.get_device_error() == 0


FEW = [
    # cache, act, hq, hkv, d, bs: requests whose rows fit one row tile (128 / group tokens)
    (BF16, BF16, 8, 2, 128, 16), (F16, F16, 3, 1, 64, 32), (E4M3, BF16, 2, 2, 128, 32), (E4M3, F16, 24, 2, 64, 16),
]


@pytest.mark.parametrize("cfg", FEW, ids=lambda c: f"c{c[0]}a{c[1]}h{c[2]}x{c[3]}d{c[4]}bs{c[5]}")
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 1), (70, 130), (300, 0), (5000, 7)])
def test_extend_of_few_rows(cfg, window, sinks):
    cache, act, hq, hkv, d, bs = cfg
    for rows, prefix in (([1, 5, 0, 9], [300, 0, 17, 640]), ([10], [1500]), ([3] * 12, list(range(0, 480, 40)))):
        c = Case(cache, act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows) + window)
        q = c.rows(sum(rows), hq).cuda()
        give_back(c, prefix, window, sinks)
        c.cuda()
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks)
        assert pkv.get_device_error() == 0
        ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, window, sinks)
        check_attention(out, lse, ref, act, d, f"{cfg} {window} {sinks} {rows}")


@pytest.mark.parametrize("rows,hint", [(40, 20), (200, 20), (200, 64), (3, 2)])
def test_extend_reports_rows_beyond_the_hint(rows, hint):
    # 4 heads per kv head: row tiles of 32 tokens.  Rows beyond the hint are reported or computed,
    # never left out silently; the other request is computed
    c = Case(BF16, BF16, 1, 64, 16, [10 + rows, 60], seed=14).cuda()
    q = c.rows(rows + 2, 4).cuda()
    out = torch.full_like(q, float("nan"))
    pkv.paged_extend_attn_window(c.k, c.v, q, out, ints([0, rows, rows + 2]), ints([10, 58]), c.bt, 0.125, hint,
                                 10 + rows, 30, 2)
    err = pkv.get_device_error()
    done = ~torch.isnan(out).any(-1).any(-1)
    assert bool(done[:hint].all()) and bool(done[rows:].all())
    assert err == (0 if bool(done.all()) else 3)
    ref = R.attention(*c.values(), to_f64(q), [0, rows, rows + 2], [10, 58], c.tables, 4, 0.125, 30, 2)[0]
    assert np.abs(to_f64(out) - ref)[done.cpu().numpy()].max() < 0.05


@pytest.mark.parametrize("at", [0, 37, 69])
def test_extend_of_a_prompt_among_single_tokens(at):
    # one long request among many of a row or none: blocks are counted by rows
    rows, prefix = [1] * 70, [(7 * i) % 90 for i in range(70)]
    for i in (3, 4, 36, 38):
        rows[i] = 0
    rows[at], prefix[at] = 600, 40
    c = Case(BF16, BF16, 2, 64, 16, [p + n for p, n in zip(prefix, rows)], seed=13).cuda()
    q = c.rows(sum(rows), 8).cuda()
    out, lse = run_extend(c, q, 8, rows, prefix, 100, 3)
    ref = R.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, 8, 1 / 8, 100, 3)
    check_attention(out, lse, ref, BF16, 64)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("cache,act", [(F16, F16), (E4M3, BF16)])
def test_extend_of_a_whole_window_is_the_plain_extend(cache, act):
    prefix, rows = [300, 0], [90, 200]
    c = Case(cache, act, 2, 128, 16, [390, 200], seed=5).cuda()
    q = c.rows(290, 8).cuda()
    plain = torch.empty_like(q)
    pkv.paged_extend_attn(c.k, c.v, q, plain, ints([0, 90, 290]), ints(prefix), c.bt, 1 / 128 ** 0.5, 200, 390,
                          k_scale=c.k_scale, v_scale=c.v_scale)
    for window, sinks in ((390, 0), (2**31 - 1, 9)):
        out, _ = run_extend(c, q, 8, rows, prefix, window, sinks)
        # (its keys may be split: both round their weights, by 2^-11 of the values, and the output)
        vmax = float(np.abs(c.values()[1]).max())
        assert torch.allclose(out.float(), plain.float(), rtol=torch.finfo(TDT[act]).eps, atol=2 * 2.0 ** -11 * vmax)


def test_extend_reports_and_leaves_alone():
    c = Case(F16, F16, 1, 64, 16, [96, 96], seed=6).cuda()
    q = c.rows(20, 4).cuda()
    for prefix in ([-1, 50], [90, 50]):                        # negative, past the table
        out, _ = run_extend(c, q, 4, [10, 10], prefix, 8, 2)
        assert pkv.get_device_error() == 3
        assert bool(torch.isnan(out[:10]).all()) and bool(torch.isfinite(out[10:]).all())
    c.bt[1, 3] = -1                                            # a block that rows of request 1 see
    out, _ = run_extend(c, q, 4, [10, 10], [50, 50], 8, 2)
    assert pkv.get_device_error() == 1 and bool(torch.isfinite(out).all())


def test_decode_and_extend_of_a_window_in_a_cuda_graph():
    c = Case(BF16, BF16, 2, 128, 16, [400, 90], seed=7).cuda()
    q, qd = c.rows(60, 8).cuda(), c.rows(2, 8).cuda()
    out, dec = torch.empty_like(q), torch.empty_like(qd)
    qi, pl, n = ints([0, 40, 60]), ints([360, 70]), ints([400, 90])
    ws = torch.empty(pkv.extend_widen_workspace_bytes(c.k), dtype=torch.uint8, device="cuda")
    dws = torch.empty(pkv.decode_window_workspace_bytes(c.k, 2, 8, 400, 100, 4, 4), dtype=torch.uint8, device="cuda")

    def step():
        pkv.paged_extend_attn_window(c.k, c.v, q, out, qi, pl, c.bt, 0.1, 40, 400, 100, 4, workspace=ws)
        pkv.paged_decode_attn_window(c.k, c.v, qd, dec, c.bt, n, 0.1, 400, 100, 4, num_splits=4, workspace=dws)

    step()
    want = out.clone(), dec.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(2):
        out.fill_(float("nan"))
        dec.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dec, want[1])
    assert pkv.get_device_error() == 0

"""GPU checks of the extend kernels that long chunks run on, in a window and over block scales: items
taken as they come (several with rows for every SM, counted by the length hint and by the rows),
pages widened into the workspace, and half tiles.  Sizes follow the device's SM count; where a tracer is
to be had, each test also says which kernels ran."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests import paths_testlib as P
from tests.pkv_testlib import BF16, E4M3, F16, to_f64
from tests.scaled_testlib import SCALED, TDT, Case, check_attention, ints

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


class Call:
    """An extend call: `rows` of queries after `prefix` tokens, in a window and / or over block scales,
    blocks that no row sees given back."""

    def __init__(self, cache, act, hq, hkv, d, bs, rows, prefix, window, sinks, seed, width=None):
        self.c = c = Case(cache, act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=seed, width=width)
        self.hq, self.rows, self.prefix, self.window, self.sinks = hq, rows, prefix, window, sinks
        self.seen = set()                            # blocks that hold a token some row may see
        nan = 0x7F if c.k.dtype == torch.uint8 else float("nan")
        for b, (p, n) in enumerate(zip(prefix, rows)):
            for lb in range(-(-(p + n) // bs)):
                t = lb * bs + np.arange(bs)
                blk = int(c.tables[b, lb])
                gone = (t >= sinks) & (t < p - window + 1) if window else np.zeros(bs, bool)
                gone |= t >= p + n
                for off in np.flatnonzero(gone):
                    c.k[blk, :, off], c.v[blk, :, off] = nan, nan
                if window and (gone & (t < p + n)).sum() == bs:
                    c.tables[b, lb] = -1 if lb % 2 else c.k.shape[0] + 5
                elif n:
                    self.seen.add(blk)
        self.ip = [0] + [int(i) for i in np.cumsum(rows)]
        self.q = c.rows(self.ip[-1], hq).cuda()
        c.cuda()
        self.need = pkv.extend_block_scaled_workspace_bytes(c.k) if cache == SCALED else pkv.extend_widen_workspace_bytes(c.k)
        self.layout = ints(self.ip), ints(prefix)

    def run(self, fill=None):
        """out, lse and the workspace (of bytes `fill`, or none)."""
        c, q = self.c, self.q
        out = torch.full((q.shape[0] + 1, self.hq, c.d), 7.0, dtype=TDT[c.act], device="cuda")
        lse = torch.full((q.shape[0] + 1, self.hq), 7.0, device="cuda")
        ws = None if fill is None else torch.full((self.need,), fill, dtype=torch.uint8, device="cuda")
        args = (q, out[:-1], *self.layout, c.bt, 1 / c.d ** 0.5, max(self.rows),
                max(p + n for p, n in zip(self.prefix, self.rows)))
        if c.cache == SCALED:
            pkv.paged_extend_attn_block_scaled(c.k, c.v, c.ks, c.vs, *args, window=self.window, sink_tokens=self.sinks,
                                               lse_out=lse[:-1], workspace=ws)
        else:
            pkv.paged_extend_attn_window(c.k, c.v, *args, self.window, self.sinks, k_scale=c.k_scale, v_scale=c.v_scale,
                                         lse_out=lse[:-1], workspace=ws)
        assert pkv.get_device_error() == 0
        assert bool((out[-1] == 7.0).all()) and bool((lse[-1] == 7.0).all())
        return out[:-1], lse[:-1], ws

    def reference(self):
        c = self.c
        return P.attention(*c.values(), to_f64(self.q), self.ip, self.prefix, c.tables, self.hq, 1 / c.d ** 0.5,
                           self.window, self.sinks)

    def claimed(self, ws):
        """The blocks that a call with a workspace widened (the list behind the two pools)."""
        nb = self.c.k.shape[0]
        at = self.need - -(-(1 + 2 * nb) * 4 // 256) * 256
        words = ws[at:].view(torch.int32).cpu().numpy()
        return [int(i) for i in words[1 + nb:1 + nb + int(words[0])]]

    def check(self, out, lse, what=""):
        check_attention(out, lse, self.ref, self.c.act, self.c.d, what)

    def run_twice(self, fill=None):
        """run(), checked; once more for the same bits and the kernels that ran."""
        self.ref = self.reference()
        out, lse, ws = self.run(fill)
        self.check(out, lse, f"{fill}")
        (again, lse2, _), ran = P.profiled(lambda: self.run(None if fill is None else 255 - fill))
        assert torch.equal(again, out) and torch.equal(lse2, lse)
        return ws, ran


def form(ran):
    """What the one extend kernel of a call was: head dim, cache, act, then its flags."""
    (a,) = ran["extend_kernel"]
    names = ["hd", "cache", "act", "prefix", "shared", "window", "scaled", "split", "take", "half"]
    assert len(a) == len(names)
    return dict(zip(names, a))


# cache, act, d, bs, window, sinks
KINDS = [(BF16, BF16, 128, 16, 150, 5), (F16, F16, 64, 32, 100, 0), (E4M3, F16, 128, 32, 70, 20), (E4M3, BF16, 64, 16, 4096, 0),
         (SCALED, BF16, 128, 16, 0, 0), (SCALED, F16, 64, 32, 0, 0), (SCALED, BF16, 64, 16, 90, 3), (SCALED, F16, 128, 32, 130, 0)]
IDS = [f"c{k[0]}a{k[1]}d{k[2]}bs{k[3]}w{k[4]}" for k in KINDS]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_items_taken_as_they_come(kind):
    # 16 query rows a token: pairs of 16 tokens; 4 items with rows for every SM, of 1 to 4 key tiles,
    # of nearly equal requests (counted by the length hint), a part of them past their rows
    cache, act, d, bs, window, sinks = kind
    hkv, batch = 8, 10
    pairs = max(2, -(-4 * sms() // (hkv * batch)))
    rng = np.random.default_rng(d + bs)
    rows = [int(n) for n in 16 * pairs - rng.integers(0, 20, batch)]
    rows[3], rows[7] = 16 * pairs, 0
    prefix = [int(n) for n in rng.integers(0, 300, batch)]
    call = Call(cache, act, 16 * hkv, hkv, d, bs, rows, prefix, window, sinks, seed=d)
    assert sum(-(-n // 16) for n in rows) * hkv >= 3 * sms() and pairs < 16
    _, ran = call.run_twice()
    if ran:
        f = form(ran)
        assert (f["take"], f["split"], f["half"]) == (1, 0, 0), f
        assert (f["window"], f["scaled"]) == (int(window > 0), int(cache == SCALED))


def uneven(hkv, long, group):
    """Rows and prefixes of a few long requests among many of a row, three or none, the items of the
    long ones at least three for every SM."""
    rng = np.random.default_rng(long)
    pair = 2 * (128 // group)
    batch_long = -(-3 * sms() // (hkv * -(-long // pair)))
    rows = [int(long - i % 5) for i in range(batch_long)] + [[1, 3, 0][i % 3] for i in range(8 * batch_long)]
    order = rng.permutation(len(rows))
    return [rows[i] for i in order], [int(n) for n in rng.integers(0, 250, len(rows))]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_items_counted_by_rows(kind):
    cache, act, d, bs, window, sinks = kind
    rows, prefix = uneven(8, 160, 16)
    call = Call(cache, act, 128, 8, d, bs, rows, prefix, window, sinks, seed=d + 1)
    _, ran = call.run_twice()
    if ran:
        f = form(ran)
        assert (f["take"], f["split"], f["half"]) == (2, 0, 0), f


# widened: bf16 (V), fp8 of one scale per tensor, and block-scaled caches
WIDE = [(BF16, BF16, 128, 16, 150, 5), (BF16, BF16, 64, 32, 4096, 0), (E4M3, F16, 64, 32, 70, 20), (E4M3, BF16, 128, 16, 100, 0),
        (SCALED, BF16, 128, 16, 0, 0), (SCALED, F16, 64, 32, 0, 0), (SCALED, BF16, 64, 32, 90, 3), (SCALED, F16, 128, 16, 130, 0)]
WIDE_IDS = [f"c{k[0]}a{k[1]}d{k[2]}bs{k[3]}w{k[4]}" for k in WIDE]


def check_widened(call, take):
    ws, ran = call.run_twice(0xFF)
    got = call.claimed(ws)
    assert len(set(got)) == len(got) and call.seen <= set(got)      # every block that a row sees, once
    assert all(0 <= blk < call.c.k.shape[0] for blk in got)
    if call.window:
        hidden = {int(t) for b, n in enumerate(call.rows) for t in call.c.tables[b] if n} - call.seen
        assert not hidden & set(got)                                # and none that no row sees
    if ran:
        f = form(ran)
        cache = 3 if call.c.act == BF16 else F16
        assert (f["take"], f["split"], f["half"], f["cache"], f["scaled"]) == (take, 0, 0, cache, 0), f
        assert len(ran["claim_kernel"]) == 1
    # the codes, without a workspace
    out, lse, _ = call.run()
    call.check(out, lse, "codes")


@pytest.mark.parametrize("kind", WIDE, ids=WIDE_IDS)
def test_widened_pages(kind):
    # 32 query rows a token: pairs of 8 tokens, 16 of them a request, as many as give each SM 3 items
    cache, act, d, bs, window, sinks = kind
    hkv, rng = 2, np.random.default_rng(d)
    batch = -(-3 * sms() // (hkv * 16)) + 2
    rows = [128 - int(n) for n in rng.integers(0, 8, batch)]
    rows[0], rows[batch - 1] = 128, 0
    prefix = [int(n) for n in rng.integers(0, 300, batch)]
    call = Call(cache, act, 32 * hkv, hkv, d, bs, rows, prefix, window, sinks, seed=bs)
    # a prefix block that two requests share
    if not window:
        call.seen.discard(int(call.c.tables[2, 0]))
        call.c.tables[2, 0] = call.c.tables[1, 0]
        call.c.bt = torch.from_numpy(call.c.tables).cuda()
    check_widened(call, 1)


@pytest.mark.parametrize("kind", WIDE, ids=WIDE_IDS)
def test_widened_pages_of_items_counted_by_rows(kind):
    cache, act, d, bs, window, sinks = kind
    rows, prefix = uneven(4, 130, 32)
    check_widened(Call(cache, act, 128, 4, d, bs, rows, prefix, window, sinks, seed=bs + 1), 2)


@pytest.mark.parametrize("cache,act,d,bs", [(BF16, BF16, 128, 16), (F16, F16, 64, 32), (E4M3, BF16, 128, 32), (E4M3, F16, 64, 16),
                                            (SCALED, BF16, 64, 16), (SCALED, F16, 128, 32), (BF16, BF16, 64, 16)])
@pytest.mark.parametrize("per,splits", [(0.05, 8), (0.2, 4), (0.46, 2), (0.92, 1)])
def test_half_tiles_in_a_window(cache, act, d, bs, per, splits):
    # requests of 1 to 32 rows (4 heads: one row tile) over long windows; `per` items for every SM
    hkv, rng = 2, np.random.default_rng(d + splits)
    batch = max(2, int(per * sms()) // hkv)
    rows = [int(n) for n in rng.integers(0, 4, batch)]
    rows[0], rows[-1] = 32, 1
    prefix = [int(n) for n in rng.integers(0, 4000, batch)]
    prefix[0] = 4068
    window, sinks = 4000, 9
    call = Call(cache, act, 4 * hkv, hkv, d, bs, rows, prefix, window, sinks, seed=splits)
    _, ran = call.run_twice()
    if ran:
        f = form(ran)
        assert (f["half"], f["split"], f["window"], f["scaled"]) == (1, 1, 1, int(cache == SCALED)), f


@pytest.mark.parametrize("act", [BF16, F16])
@pytest.mark.parametrize("rows,prefix", [([20], [900]), ([140], [0]), ([3, 0, 40], [100, 9, 0])])
def test_values_under_small_scales(act, rows, prefix):
    # V takes part as f16: under scales of 2^-30 to 2^-16 its steps are 2^-24, whatever the code, so
    # that each value is off by 2^-25 at most, which the bound's last term holds
    c = Case(SCALED, act, 2, 64, 16, [p + n for p, n in zip(prefix, rows)], seed=3)
    c.vs = torch.from_numpy(np.exp2(c.rng.integers(-30, -15, c.vs.shape)).astype(np.float32))
    c.cuda()
    q = c.rows(sum(rows), 8).cuda()
    ip = [0] + [int(i) for i in np.cumsum(rows)]
    ref = P.attention(*c.values(), to_f64(q), ip, prefix, c.tables, 8, 1 / 8)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    pkv.paged_extend_attn_block_scaled(c.k, c.v, c.ks, c.vs, q, out, ints(ip), ints(prefix), c.bt, 1 / 8, max(rows),
                                       max(p + n for p, n in zip(prefix, rows)), lse_out=lse)
    check_attention(out, lse, ref, act, 64)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", [WIDE[0], WIDE[3], WIDE[4], WIDE[7]], ids=[WIDE_IDS[i] for i in (0, 3, 4, 7)])
def test_widened_pages_in_two_graphs_of_one_workspace(kind):
    # two captured calls, replayed in turn over one workspace, with the pools' contents changed between
    cache, act, d, bs, window, sinks = kind
    rows, prefix = [125, 128, 1, 0, 120], [40, 7, 300, 5, 0]
    calls = [Call(cache, act, 256, 8, d, bs, rows, [p + 16 * i for p in prefix], window, sinks, seed=i + d) for i in range(2)]
    ws = torch.empty(max(c.need for c in calls), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in calls:
        c, out = call.c, torch.empty_like(call.q)
        args = (call.q, out, *call.layout, c.bt, 1 / d ** 0.5, max(rows), max(p + n for p, n in zip(call.prefix, rows)))

        def step():
            if cache == SCALED:
                pkv.paged_extend_attn_block_scaled(c.k, c.v, c.ks, c.vs, *args, window=window, sink_tokens=sinks, workspace=ws)
            else:
                pkv.paged_extend_attn_window(c.k, c.v, *args, window, sinks, k_scale=c.k_scale, v_scale=c.v_scale,
                                             workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                step()
        graphs.append(graph)
        outs.append(out)
    for turn in range(3):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for call, out in zip(calls, outs):
            want, _, used = call.run(0xFF)
            assert len(call.claimed(used)) >= len(call.seen) > 0      # (these calls do widen)
            assert torch.equal(out, want)
            pools = (call.c.k, call.c.v) if cache in (F16, BF16) else (call.c.ks, call.c.vs) if cache == SCALED else (call.c.k,)
            for t in pools:
                t.mul_(0.5) if t.dtype != torch.uint8 else t.bitwise_xor_(0x80)
        torch.cuda.synchronize()
    assert pkv.get_device_error() == 0

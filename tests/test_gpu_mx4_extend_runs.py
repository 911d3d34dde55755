"""GPU checks of the extend over microscaled codes in runs of key tiles, cut on the device by the requests'
lengths: items of one part and of many, rows of none to several tiles, windows, NaN, lengths that change
under a captured graph.  Where a tracer is to be had, each test also says that this kernel ran."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests import paths_testlib as P
from tests.mx4_testlib import Mx4Case, indptr
from tests.pkv_testlib import BF16, F16, to_f64
from tests.scaled_testlib import TDT, check_attention, ints

pytestmark = pytest.mark.gpu

TAKE = 8  # of the extend kernel's template arguments: 3 is a run per CTA


class Call:
    def __init__(self, hq, hkv, d, bs, act, rows, prefix, window=0, sinks=0, most=None, longest=None):
        self.c = c = Mx4Case(act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows) + d)
        self.hq, self.rows, self.prefix, self.window, self.sinks = hq, rows, prefix, window, sinks
        for b, n in enumerate(c.lens):               # what lies behind the last token
            if n % bs:
                c.ks[int(c.tables[b, n // bs]), :, n % bs:] = 255
                c.vs[int(c.tables[b, n // bs]), :, n % bs:] = 255
        self.q = c.rows(sum(rows), hq).cuda()
        c.cuda()
        self.ip, self.pl = ints(indptr(rows)), ints(prefix)
        self.most, self.longest = most or max(rows), longest or max(c.lens)
        self.ws = torch.full((pkv.extend_mx4_workspace_bytes(c.k),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, work=True):
        """out and lse, a row longer than the call's, which stays as it is."""
        c, n = self.c, self.q.shape[0]
        out = torch.full((n + 1, self.hq, c.d), 7.0, dtype=TDT[c.act], device="cuda")
        lse = torch.full((n + 1, self.hq), 7.0, device="cuda")
        self.into(out[:-1], lse[:-1], work)
        assert bool((out[n] == 7.0).all()) and bool((lse[n] == 7.0).all())
        return out[:-1], lse[:-1]

    def into(self, out, lse, work=True):
        c = self.c
        pkv.paged_extend_attn_mx4(c.k, c.v, c.ks, c.vs, self.q, out, self.ip, self.pl, c.bt, 1 / c.d ** 0.5, self.most,
                                  self.longest, window=self.window, sink_tokens=self.sinks, lse_out=lse,
                                  workspace=self.ws if work else None)

    def ref(self):
        return P.attention(*self.c.values(), to_f64(self.q), indptr(self.rows), self.prefix, self.c.tables, self.hq,
                           1 / self.c.d ** 0.5, self.window, self.sinks)


def in_runs(call):
    result, ran = P.profiled(call)
    assert ran is None or ([a[TAKE] for a in ran["extend_kernel"]] == [3] and "merge_runs_kernel" in ran), ran
    return result


CALLS = [
    # hq, hkv, d, bs, act, rows, prefix, window, sinks
    (8, 2, 128, 16, BF16, [100], [5000], 0, 0),                                         # parts of two tiles
    (16, 2, 64, 32, F16, [40, 9, 0, 33, 20], [300, 3000, 50, 1500, 0], 0, 0),
    (8, 1, 128, 32, F16, [20, 1] * 25, list(range(1, 4001, 80)), 0, 0),                 # units over two warps' worth
    (8, 2, 64, 16, BF16, [100, 90], [8000, 300], 6000, 130),
    (8, 2, 128, 16, BF16, [100, 90, 1], [8000, 300, 6500], 6000, 0),
    (32, 8, 128, 16, BF16, [91, 77, 95, 43, 0, 32, 58, 31], [2052, 2107, 2280, 977, 2296, 962, 2029, 780], 0, 0),
    (3, 1, 128, 16, F16, [100], [9000], 0, 0),                                          # a tile a part
]


@pytest.mark.parametrize("cfg", CALLS, ids=lambda c: f"h{c[0]}x{c[1]}-d{c[2]}-b{len(c[5])}-w{c[7]}")
def test_runs(cfg):
    call = Call(*cfg)
    ref = call.ref()
    for work in (True, False):
        out, lse = in_runs(call.run) if work else call.run(False)
        check_attention(out, lse, ref, call.c.act, call.c.d, f"{work}")
        again, _ = call.run(work)
        assert torch.equal(out, again)
    assert pkv.get_device_error() == 0


def test_nan_in_one_part():
    call = Call(8, 2, 128, 16, BF16, [100], [5000])
    good, _ = call.run()
    call.c.vs[int(call.c.tables[0, 100]), 0, 3, 2] = 255       # V of one key, dims 64 .. 95, heads 0 .. 3
    out, lse = in_runs(call.run)
    assert bool(torch.isnan(out[:, :4, 64:96]).all()) and torch.equal(out[:, 4:], good[:, 4:])
    assert torch.equal(out[:, :4, :64], good[:, :4, :64]) and bool(torch.isfinite(lse).all())
    call.c.ks[int(call.c.tables[0, 50]), 1, 0, 0] = 255        # K of one key: every row of heads 4 .. 7
    call.q[17, 1] = float("nan")
    out, lse = call.run()
    assert bool(torch.isnan(out[:, 4:]).all()) and bool(torch.isnan(lse[:, 4:]).all())
    assert bool(torch.isnan(out[17, 1]).all()) and bool(torch.isfinite(lse[:17, :4]).all())
    assert bool(torch.isfinite(lse[18:, :4]).all()) and torch.equal(out[:17, :4, :64], good[:17, :4, :64])
    assert pkv.get_device_error() == 0


def test_lengths_that_change_under_a_graph():
    rows, long = [60, 33, 1, 64], [4000, 3500, 200, 10]
    call = Call(8, 2, 128, 16, BF16, rows, long)
    out, lse = torch.empty_like(call.q), torch.empty((call.q.shape[0], 8), device="cuda")
    call.into(out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.into(out, lse)
    for prefix in (long, [0, 100, 4060, 900], [10, 4000, 0, 64]):
        prefix = [min(p, n) for p, n in zip(prefix, long)]     # (each within its own table)
        call.pl.copy_(ints(prefix))
        call.prefix = prefix
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        check_attention(out, lse, call.ref(), BF16, 128, f"{prefix}")
    assert pkv.get_device_error() == 0


def test_reports():
    rows, prefix = [60, 33, 1, 64], [4000, 3500, 200, 10]
    call = Call(8, 2, 128, 16, BF16, rows, prefix)
    good, _ = call.run()
    call.pl.copy_(ints([4000, -5, 200, 10]))                   # a request that cannot be: the others as they were
    out, _ = call.run()
    keep = torch.ones(158, dtype=torch.bool)
    keep[60:93] = False
    assert pkv.get_device_error() == 3 and torch.equal(out[keep.cuda()][:60], good[:60]) and torch.equal(out[93:], good[93:])
    call.pl.copy_(ints(prefix))
    call.c.bt[0, 7] = call.c.k.shape[0]                        # a block outside the pool reads zeros
    out, _ = call.run()
    assert pkv.get_device_error() == 1 and torch.equal(out[60:], good[60:]) and bool(torch.isfinite(out[:60]).all())
    call.ip.copy_(ints([0, 60, 400, 401, 465]))                # rows that the call does not have
    out, _ = call.run()
    assert pkv.get_device_error() != 0

"""GPU checks of NaN in extend calls through a window or over block scales: what a row sees as NaN
comes out as NaN, and what no row of a work item sees does not come out."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests import paths_testlib as P
from tests.pkv_testlib import BF16, E4M3, F16, to_f64
from tests.scaled_testlib import SCALED, TDT, Case, check_attention, ints

pytestmark = pytest.mark.gpu


def extend(c, q, rows, prefix, window, sinks=0):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ip = [0] + [int(n) for n in np.cumsum(rows)]
    layout = (q, out, ints(ip), ints(prefix), c.bt, 1 / c.d ** 0.5, max(rows), max(p + n for p, n in zip(prefix, rows)))
    if c.cache == SCALED:
        pkv.paged_extend_attn_block_scaled(c.k, c.v, c.ks, c.vs, *layout, window=window, sink_tokens=sinks, lse_out=lse)
    else:
        pkv.paged_extend_attn_window(c.k, c.v, *layout, window, sinks, k_scale=c.k_scale, v_scale=c.v_scale, lse_out=lse)
    return out, lse, ip


def put_nan(c, pool, request, pos):
    pool[int(c.tables[request, pos // c.bs]), :, pos % c.bs] = 0x7F if pool.dtype == torch.uint8 else float("nan")


CACHES = [(BF16, BF16, 128, 16, 4096), (F16, F16, 64, 32, 4096), (E4M3, BF16, 64, 16, 4096), (SCALED, F16, 128, 16, 0),
          (SCALED, BF16, 64, 32, 4096)]


@pytest.mark.parametrize("cache,act,d,bs,window", CACHES)
@pytest.mark.parametrize("rows,prefix", [([9], [2100]), ([3, 5], [900, 4100]), ([70], [900]), ([40], [0])])
def test_queries_that_are_nan(cache, act, d, bs, window, rows, prefix):
    # key tiles split over clusters, in whole and in half tiles, and calls of one CTA an item
    c = Case(cache, act, 2, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
    q = c.rows(sum(rows), 8).cuda()
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    bad[0, 3] = bad[sum(rows) - 1] = bad[sum(rows) // 2, 6] = True
    # (one NaN among a query's numbers does for all of its scores)
    q[bad.cuda()] = torch.where(torch.arange(d, device="cuda") == 5, float("nan"), 1.0).to(q.dtype)
    out, lse, ip = extend(c, q, rows, prefix, window)
    assert pkv.get_device_error() == 0
    assert bool(torch.isnan(out[bad.cuda()]).all()) and bool(torch.isnan(lse[bad.cuda()]).all())
    x = to_f64(q)
    x[bad.numpy()] = 0
    ref = P.attention(*c.values(), x, ip, prefix, c.tables, 8, 1 / d ** 0.5, window)
    ok = ~bad.numpy()
    ref = (ref[0][ok], ref[1][ok], {k: v[ok] for k, v in ref[2].items()})
    check_attention(out[torch.from_numpy(ok).cuda()], lse[torch.from_numpy(ok).cuda()], ref, act, d)


@pytest.mark.parametrize("cache,act,d,bs,window", CACHES)
def test_a_key_that_is_nan_alone_in_its_part(cache, act, d, bs, window):
    # 897 keys are eight key tiles; where eight CTAs share them the last one has key 896 alone
    c = Case(cache, act, 2, d, bs, [897, 897], seed=d).cuda()
    q = c.rows(2, 8).cuda()
    put_nan(c, c.k, 0, 896)
    out, lse, ip = extend(c, q, [1, 1], [896, 896], window)
    assert pkv.get_device_error() == 0
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    ref = P.attention(*c.values(), to_f64(q), ip, [896, 896], c.tables, 8, 1 / d ** 0.5, window)
    ref = (ref[0][1:], ref[1][1:], {k: v[1:] for k, v in ref[2].items()})
    check_attention(out[1:], lse[1:], ref, act, d)


@pytest.mark.parametrize("cache,act,d,bs", [(BF16, BF16, 128, 16), (BF16, BF16, 64, 32), (F16, F16, 128, 32),
                                            (E4M3, BF16, 64, 16), (E4M3, F16, 128, 16), (SCALED, BF16, 128, 16),
                                            (SCALED, F16, 64, 32)])
@pytest.mark.parametrize("prefix,window,sinks", [(37, 4096, 0), (46, 50, 3), (1005, 4096, 0), (990, 300, 7)])
def test_values_of_later_tokens_that_no_row_of_an_item_sees(cache, act, d, bs, prefix, window, sinks):
    # 4 heads a kv head: items of 64 rows.  The token after the first item's last one lies in that
    # one's 16 tokens: its V (NaN) is the second item's alone, whose rows all see it
    c = Case(cache, act, 2, d, bs, [prefix + 90], seed=prefix).cuda()
    assert (prefix + 64) % 16
    q = c.rows(90, 8).cuda()
    put_nan(c, c.v, 0, prefix + 64)
    out, lse, ip = extend(c, q, [90], [prefix], window, sinks)
    assert pkv.get_device_error() == 0
    vals = c.values()
    vals[1] = np.nan_to_num(vals[1])
    ref = P.attention(*vals, to_f64(q), ip, [prefix], c.tables, 8, 1 / d ** 0.5, window, sinks)
    ref = (ref[0][:64], ref[1][:64], {k: v[:64] for k, v in ref[2].items()})
    check_attention(out[:64], lse[:64], ref, act, d)
    assert bool(torch.isnan(out[64:]).all())

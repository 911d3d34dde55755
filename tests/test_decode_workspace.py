"""The workspace of the decode calls through a window or over block scales: sized once for the
largest batch and length, it serves every smaller one."""
import ctypes
import random

import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from paged_kv_cache_285_gb300 import build as pkv_build
from tests.pkv_testlib import BF16
from tests.scaled_testlib import SCALED, Case, ints
from tests.test_abi import _desc


@pytest.fixture(scope="module")
def need():
    pkv_build.build()
    lib = pkv.load()

    def f(desc, batch, hq, most, window=0, sinks=0):
        return lib.pkv_decode_window_workspace_bytes(ctypes.byref(desc), batch, hq, most, window, sinks, 0)
    return f


def test_it_never_falls(need):
    d = _desc(cache_dtype=2)
    # plans of one split or of clusters beside plans with partials
    assert need(d, 4, 8, 4096) <= need(d, 400, 8, 4096) <= need(d, 512, 8, 4096)
    rng = random.Random(5)
    for _ in range(400):
        d = _desc(cache_dtype=rng.choice([1, 2]), head_dim=rng.choice([64, 128]), num_kv_heads=rng.choice([1, 2, 8]))
        hq = d.num_kv_heads * rng.choice([1, 4, 12])
        batch, most = (int(2 ** rng.uniform(0, e)) for e in (11, 20))
        window, sinks = rng.choice([(0, 0), (1, 0), (500, 3), (4096, 64), (2 ** 31 - 1, 7)])
        large = need(d, batch, hq, most, window, sinks)
        for _ in range(20):
            b, n = rng.randint(1, batch), rng.randint(0, most)
            assert need(d, b, hq, n, window, sinks) <= large, (batch, most, b, n, window, sinks)


def test_it_is_not_out_of_proportion(need):
    # at most eight partials a request and head, and those of two rounds of CTAs
    d = _desc(cache_dtype=2, head_dim=128, num_kv_heads=8)
    for batch in (1, 100, 5000):
        rows = 8 * batch + 2 * 4 * 152 // 8 + 1
        assert need(d, batch, 32, 2 ** 20) <= rows * 32 * (128 + 1) * 4 + 256
    assert need(d, 5000, 32, 64) == 0       # one split whatever the batch
    assert need(d, 0, 32, 1000) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,window,sinks", [(128, 0, 0), (64, 0, 0), (128, 4000, 9)])
def test_sized_for_the_largest_it_serves_every_smaller(d, window, sinks):
    batch, hq, hkv, most = 96, 4, 2, 6000
    c = Case(SCALED, BF16, hkv, d, 16, [most] * 3, seed=d).cuda()
    c.tables = c.tables[[i % 3 for i in range(batch)]]
    bt = torch.from_numpy(c.tables).cuda()
    q = c.rows(batch, hq).cuda()
    size = pkv.decode_window_workspace_bytes(c.k, batch, hq, most, window, sinks)
    ws = torch.full((size + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    seen = set()
    for b in (1, 2, 5, 16, 30, 40, 64, 76, 77, 96):
        for n in (1, 64, 65, 200, 700, 1000, 2048, 5999, 6000):
            lens = ints([max(n - 37 * i, 1) for i in range(b)])
            out, one = torch.empty_like(q[:b]), torch.empty_like(q[:b])
            args = (c.k, c.v, c.ks, c.vs, q[:b])
            pkv.paged_decode_attn_block_scaled(*args, out, bt[:b], lens, 1 / d ** 0.5, n, window, sinks, workspace=ws[:size])
            pkv.paged_decode_attn_block_scaled(*args, one, bt[:b], lens, 1 / d ** 0.5, n, window, sinks, num_splits=1)
            # (both round weights by 2^-11 of the values, and the output)
            vmax = float((c.vs.max() * 448).item())
            assert torch.allclose(out.float(), one.float(), rtol=2.0 ** -7, atol=2 * 2.0 ** -11 * vmax), (b, n)
            seen.add(bool((ws[:size] != 0xAB).any()))
    assert True in seen and bool((ws[size:] == 0xAB).all()) and pkv.get_device_error() == 0

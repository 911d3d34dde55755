"""GPU checks of the decode forms of few and of many requests (splits joined in clusters, splits of
falling length) for every kind of cache in a window, and of a server's step in a graph and on two
streams, its log-sum-exps and pools included."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from tests import paths_testlib as P
from tests.pkv_testlib import BF16, E4M3, F16, to_f64
from tests.scaled_testlib import SCALED, TDT, Case, check_attention, ints

pytestmark = pytest.mark.gpu


def decode(c, q, hq, lens, window, sinks):
    n, most = len(lens), max(lens)
    out = torch.full((n, hq, c.d), float("nan"), dtype=TDT[c.act], device="cuda")
    lse = torch.full((n, hq), float("nan"), device="cuda")
    need = pkv.decode_window_workspace_bytes(c.k, n, hq, most, window, sinks)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    args = (q, out, c.bt, ints(lens), 1 / c.d ** 0.5, most)
    if c.cache == SCALED:
        pkv.paged_decode_attn_block_scaled(c.k, c.v, c.ks, c.vs, *args, window=window, sink_tokens=sinks, lse_out=lse,
                                           workspace=ws)
    else:
        pkv.paged_decode_attn_window(c.k, c.v, *args, window, sinks, k_scale=c.k_scale, v_scale=c.v_scale, lse_out=lse,
                                     workspace=ws)
    return out, lse


def check(cache, act, hq, hkv, d, bs, lens, window, sinks):
    """A decode whose hidden tokens are NaN; the kernels that ran."""
    c = Case(cache, act, hkv, d, bs, lens, seed=sum(lens) % 1009)
    nan = 0x7F if c.k.dtype == torch.uint8 else float("nan")
    for b, n in enumerate(lens):
        t = np.arange(c.tables.shape[1] * bs)
        gone = (t >= n) | ((t >= sinks) & (t < n - window)) if window else t >= n
        for lb in range(-(-n // bs)):
            here = gone[lb * bs:(lb + 1) * bs]
            blk = int(c.tables[b, lb])
            for off in np.flatnonzero(here):
                c.k[blk, :, off], c.v[blk, :, off] = nan, nan
            if here.all():
                c.tables[b, lb] = -1
    q = c.rows(len(lens), hq).cuda()
    c.cuda()
    (out, lse), ran = P.profiled(lambda: decode(c, q, hq, lens, window, sinks))
    assert pkv.get_device_error() == 0
    ref = P.attention(*c.values(), to_f64(q), range(len(lens) + 1), [n - 1 for n in lens], c.tables, hq, 1 / d ** 0.5,
                      window, sinks)
    check_attention(out, lse, ref, act, d, f"{cache} {window}")
    return ran


def form(ran):
    (a,) = ran["decode_kernel"]
    names = ["hd", "cache", "act", "warps", "stages", "cascade", "window", "scaled", "joined"]
    assert len(a) == len(names)
    return dict(zip(names, a))


KINDS = [(F16, F16, 128, 16), (F16, F16, 64, 32), (BF16, BF16, 64, 16), (E4M3, F16, 128, 32), (E4M3, BF16, 64, 16),
         (SCALED, BF16, 128, 16), (SCALED, F16, 64, 32)]


@pytest.mark.parametrize("cache,act,d,bs", KINDS)
@pytest.mark.parametrize("lens,window,sinks", [([700, 33, 1, 0], 600, 5), ([1200], 1000, 0), ([900, 4000, 17], 300, 130),
                                               ([2000, 2, 1999], 4096, 0)])
def test_few_requests_in_a_window(cache, act, d, bs, lens, window, sinks):
    ran = check(cache, act, 8, 2, d, bs, lens, window, sinks)
    if ran:
        f = form(ran)
        assert (f["joined"], f["window"], f["scaled"]) == (1, 1, int(cache == SCALED)), f
        assert "merge_kernel" not in ran


@pytest.mark.parametrize("act,hq,hkv,d,bs,window,sinks", [(BF16, 2, 2, 128, 16, 3590, 33), (F16, 8, 2, 128, 32, 5000, 0),
                                                          (BF16, 2, 2, 64, 16, 7100, 20)])
def test_many_requests_over_block_scales_in_a_window(act, hq, hkv, d, bs, window, sinks):
    # splits of falling length: most requests short, some as long as the window, some longer
    batch, rng = 80, np.random.default_rng(window)
    long = [window, window + 1, window + 17, window + sinks + 700, window - 16, 16 * (window // 32), 16 * (window // 64) + 1]
    lens = [int(n) for n in rng.permutation(long + [0, 1] + list(rng.integers(0, 90, batch - len(long) - 2)))]
    ran = check(SCALED, act, hq, hkv, d, bs, lens, window, sinks)
    if ran:
        f = form(ran)
        assert (f["joined"], f["window"], f["scaled"]) == (0, 1, 1) and len(ran["merge_kernel"]) == 1, f


def test_a_step_in_a_graph_and_on_two_streams_with_its_lse():
    hq, hkv, d, bs, act = 8, 2, 128, 16, BF16
    lens = [40, 300, 7]

    class Server:
        def __init__(self):
            self.c = c = Case(SCALED, act, hkv, d, bs, [n + 16 for n in lens], seed=32).cuda()
            self.kn, self.vn, self.q = c.rows(3, hkv).cuda(), c.rows(3, hkv).cuda(), c.rows(3, hq).cuda()
            self.qi, self.at, self.n = ints([0, 1, 2, 3]), ints(lens), ints([m + 1 for m in lens])
            self.out = torch.empty_like(self.q)
            self.lse = torch.full((3, hq), float("nan"), device="cuda")
            need = pkv.decode_window_workspace_bytes(c.k, 3, hq, 512, 0, 0, 4)
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def step(self, stream=None):
            c = self.c
            pkv.kv_append_block_scaled(c.k, c.v, c.ks, c.vs, self.kn, self.vn, self.qi, self.at, c.bt, 1, stream=stream)
            pkv.paged_decode_attn_block_scaled(c.k, c.v, c.ks, c.vs, self.q, self.out, c.bt, self.n, 1 / d ** 0.5, 512,
                                               num_splits=4, lse_out=self.lse, workspace=self.ws, stream=stream)

        def state(self):
            return self.out, self.lse, self.c.k, self.c.v, self.c.ks, self.c.vs

    one, two, graphed = Server(), Server(), Server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            graphed.step()
    for i in range(10):
        one.step()
        two.step(stream=side)
        graph.replay()
        torch.cuda.synchronize()
        for other in (two, graphed):
            for a, b in zip(one.state(), other.state()):
                assert torch.equal(a, b)
        ref = R.attention(*one.c.values(), to_f64(one.q), range(4), [n + i for n in lens], one.c.tables, hq, 1 / d ** 0.5)
        check_attention(one.out, one.lse, ref, act, d, f"step {i}")
        for s in (one, two, graphed):
            s.at += 1
            s.n += 1
            s.lse.fill_(float("nan"))
        torch.cuda.synchronize()
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("cache,act,d,bs", KINDS)
@pytest.mark.parametrize("lens", [[700, 33, 1], [20, 40, 64], [700, 300, 9] + [50] * 77])
def test_nan_comes_out_as_nan(cache, act, d, bs, lens):
    # a query that is NaN, and a key and a value of a visible token that are: their rows' outputs
    # alone are NaN, in clusters, with partials and in one split
    c = Case(cache, act, 2, d, bs, lens, seed=len(lens))
    bad = 0x7F if c.k.dtype == torch.uint8 else float("nan")
    at = lens[1] // 2
    c.k[int(c.tables[1, at // bs]), 0, at % bs] = bad        # request 1, kv head 0
    c.v[int(c.tables[1, at // bs]), 1, at % bs] = bad        # request 1, kv head 1
    q = c.rows(len(lens), 8)
    q[2, 5, 7] = float("nan")
    c.cuda()
    q = q.cuda()
    nan = np.zeros((len(lens), 8), bool)
    nan[1], nan[2, 5] = True, True
    for splits in (0, 1, 5):
        out, lse = (torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"))
        ws = torch.full((max(pkv.decode_window_workspace_bytes(c.k, len(lens), 8, max(lens), 4096, 0, splits), 1),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        args = (q, out, c.bt, ints(lens), 1 / d ** 0.5, max(lens))
        if cache == SCALED:
            pkv.paged_decode_attn_block_scaled(c.k, c.v, c.ks, c.vs, *args, num_splits=splits, lse_out=lse, workspace=ws)
        else:
            pkv.paged_decode_attn_window(c.k, c.v, *args, 4096, k_scale=c.k_scale, v_scale=c.v_scale, num_splits=splits,
                                         lse_out=lse, workspace=ws)
        assert pkv.get_device_error() == 0
        got = torch.isnan(out).all(-1).cpu().numpy()
        assert np.array_equal(got, nan) and np.array_equal(torch.isnan(out).any(-1).cpu().numpy(), nan)
        nan_lse = nan.copy()
        nan_lse[1, 4:] = False                               # (V does not enter it)
        assert np.array_equal(torch.isnan(lse).cpu().numpy(), nan_lse)

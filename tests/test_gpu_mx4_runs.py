"""GPU checks of the microscaled cache as it is used: prompts, forks, decoding steps and compactions in a
row, in CUDA graphs, on several streams and threads, in large pools; and the extend kernels' regimes."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import block_scaled_ref as R
from oracle import mx4_ref as M
from tests.mx4_testlib import Mx4Case, decode_ref, extend_ref, indptr, run_decode, run_extend
from tests.pkv_testlib import BF16, F16, to_f64
from tests.scaled_testlib import TDT, check_attention, ints

pytestmark = pytest.mark.gpu


def pools_of(c):
    return [t.cpu().numpy().copy() for t in (c.k, c.v, c.ks, c.vs)]


def test_a_run_of_all_calls():
    # prompts are written and attended to, one is forked (its last page copied), every branch decodes, one drops
    # half of its tokens and decodes on; after every call the pools and outputs are the reference's
    hq, hkv, d, bs, act = 8, 2, 128, 16, BF16
    c = Mx4Case(act, hkv, d, bs, [50, 23, 1], seed=21, spare=30, width=10).cuda()
    used = set(c.tables[c.tables >= 0].tolist())
    free = [i for i in range(c.k.shape[0]) if i not in used]
    set_ = pkv.KvPools([c.k, c.v, c.ks, c.vs])
    rows = [50, 23, 1]
    want = pools_of(c)

    def append(rows, at, scale=1.0):
        kn, vn = c.rows(sum(rows), hkv, scale), c.rows(sum(rows), hkv, scale)
        for i, new in enumerate((kn, vn)):
            want[i], want[i + 2] = M.append(want[i], want[i + 2], to_f64(new), indptr(rows), at, c.tables)
        pkv.kv_append_mx4(c.k, c.v, c.ks, c.vs, kn.cuda(), vn.cuda(), ints(indptr(rows)), ints(at), c.bt, max(rows))

    def same():
        for got, w in zip((c.k, c.v, c.ks, c.vs), want):
            np.testing.assert_array_equal(got.cpu().numpy(), w)

    append(rows, [0, 0, 0])
    same()
    q = c.rows(sum(rows), hq).cuda()
    out, lse = run_extend(c, q, hq, rows, [0, 0, 0])
    check_attention(out, lse, extend_ref(c, q, hq, rows, [0, 0, 0]), act, d, "prompts")
    # two branches of request 0: its full blocks shared, the last one copied for each but the first
    tables = np.full((5, 10), -1, np.int32)
    tables[:3] = c.tables
    src, dst = [], []
    for b in (3, 4):
        tables[b, :3] = c.tables[0, :3]
        tables[b, 3] = free.pop()
        src.append(c.tables[0, 3])
        dst.append(tables[b, 3])
    c.tables, c.bt = tables, torch.from_numpy(tables).cuda()
    pkv.kv_copy_blocks(set_, ints(src), ints(dst))
    for w in want:
        w[dst] = w[src]
    same()
    at = [50, 23, 1, 50, 50]
    for step in range(20):
        for b in range(5):
            if at[b] % bs == 0 and tables[b, at[b] // bs] < 0:
                tables[b, at[b] // bs] = free.pop()
        c.bt = torch.from_numpy(tables).cuda()
        append([1] * 5, at, 1.0 + 0.1 * step)
        at = [n + 1 for n in at]
        q = c.rows(5, hq).cuda()
        out, lse = run_decode(c, q, hq, at, most=100)
        check_attention(out, lse, decode_ref(c, q, hq, at), act, d, f"step {step}")
        if step == 9:  # a branch keeps its first 4 tokens and some of the others, in blocks of its own
            mine = [free.pop() for _ in range(3)]
            pkv.kv_copy_blocks(set_, ints(tables[3, :3]), ints(mine))
            for w in want:
                w[mine] = w[tables[3, :3]]
            tables[3, :3] = mine
            kept = sorted(int(x) for x in 4 + c.rng.choice(at[3] - 4, 31, replace=False))
            c.bt = torch.from_numpy(tables).cuda()
            pkv.kv_compact(set_, ints(kept), ints([0, 0, 0, 0, 31, 31]), ints([0, 0, 0, 4, 0]), c.bt, 31)
            for i in range(4):
                want[i] = M.compact(want[i], kept, [0, 0, 0, 0, 31, 31], [0, 0, 0, 4, 0], tables)
            at[3] = 35
            same()
    same()
    ko, vo = (torch.empty((sum(at), hkv, d), dtype=TDT[act], device="cuda") for _ in range(2))
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko, vo, ints(indptr(at)), ints([0] * 5), c.bt)
    for got, vals in zip((ko, vo), c.values()):
        assert np.array_equal(to_f64(got), np.concatenate([R.rows_of(vals, t, 0, m) for t, m in zip(c.tables, at)]))
    assert pkv.get_device_error() == 0


class Server:
    """A decoding step, and a compaction every now and then, over buffers of its own."""

    def __init__(self, seed=31, lens=(40, 300), hq=8, hkv=2, d=64):
        self.c = c = Mx4Case(BF16, hkv, d, 16, [n + 30 for n in lens], seed=seed).cuda()
        n = len(lens)
        self.kn, self.vn, self.q = c.rows(n, hkv).cuda(), c.rows(n, hkv).cuda(), c.rows(n, hq).cuda()
        self.qi, self.at, self.n = ints(range(n + 1)), ints(lens), ints([m + 1 for m in lens])
        self.out, self.d, self.lens = torch.empty_like(self.q), d, lens
        need = pkv.decode_mx4_workspace_bytes(c.k, n, hq, 512, 0, 0, 4)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.set = pkv.KvPools([c.k, c.v, c.ks, c.vs])
        # every third of 30 tokens moved to the front of them
        self.src = ints([m - 30 + 3 * i + 1 for m in lens for i in range(10)])
        self.ip, self.to = ints([10 * i for i in range(n + 1)]), ints([m - 30 for m in lens])
        self.pages = ints([int(c.tables[0, 0])]), ints([int(c.tables[0, -1])] if c.tables[0, -1] >= 0 else [-1])

    def step(self, stream=None):
        c = self.c
        pkv.kv_append_mx4(c.k, c.v, c.ks, c.vs, self.kn, self.vn, self.qi, self.at, c.bt, 1, stream=stream)
        pkv.paged_decode_attn_mx4(c.k, c.v, c.ks, c.vs, self.q, self.out, c.bt, self.n, self.d ** -0.5, 512, num_splits=4,
                                  workspace=self.ws, stream=stream)
        pkv.kv_compact(self.set, self.src, self.ip, self.to, c.bt, 10, stream=stream)
        pkv.kv_copy_blocks(self.set, *self.pages, stream=stream)

    def advance(self):
        self.at += 1
        self.n += 1


def test_steps_in_a_cuda_graph_and_on_two_streams():
    one, two, graphed = Server(), Server(), Server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            graphed.step()
    for i in range(10):
        before = [to_f64(one.q)] + [v.copy() for v in one.c.values()]
        one.step()
        two.step(stream=side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one.out, two.out) and torch.equal(one.out, graphed.out)
        for name in ("k", "v", "ks", "vs"):
            assert torch.equal(getattr(one.c, name), getattr(graphed.c, name)), name
            assert torch.equal(getattr(one.c, name), getattr(two.c, name)), name
        for s in (one, two, graphed):
            s.advance()
        torch.cuda.synchronize()
    # the last step's output against the reference: the pools before it, and its row
    c = one.c
    kv = before[1:]
    for i, new in enumerate((one.kn, one.vn)):
        for b, p in enumerate(n + 9 for n in one.lens):
            for g in range(c.hkv):
                codes, scales = M.quantise(to_f64(new)[b, g])
                kv[i][c.tables[b, p // 16], g, p % 16] = M.values(codes, scales)
    ref = R.attention(*kv, before[0], range(3), [n + 9 for n in one.lens], c.tables, 8, one.d ** -0.5)
    check_attention(one.out, torch.from_numpy(ref[1]), ref, BF16, one.d)
    assert pkv.get_device_error() == 0


def test_two_graphs_that_share_a_workspace():
    # a decode and an extend, each captured, replayed one after the other in one stream over the same workspace
    c = Mx4Case(F16, 2, 128, 16, [700, 1200], seed=4).cuda()
    q, qe = c.rows(2, 8).cuda(), c.rows(1190, 8).cuda()
    lens, rows, prefix = [700, 1200], [10, 1180], [690, 20]
    ws = torch.empty(max(pkv.decode_mx4_workspace_bytes(c.k, 2, 8, 1200, 0, 0, 5), pkv.extend_mx4_workspace_bytes(c.k)),
                     dtype=torch.uint8, device="cuda")
    out, oute = torch.empty_like(q), torch.empty_like(qe)
    sl, qi, pl = ints(lens), ints(indptr(rows)), ints(prefix)

    def decode():
        pkv.paged_decode_attn_mx4(c.k, c.v, c.ks, c.vs, q, out, c.bt, sl, 0.09, 1200, num_splits=5, workspace=ws)

    def extend():
        pkv.paged_extend_attn_mx4(c.k, c.v, c.ks, c.vs, qe, oute, qi, pl, c.bt, 0.09, 1180, 1200, workspace=ws)
    decode(), extend()
    want = out.clone(), oute.clone()
    graphs = []
    for fn in (decode, extend):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fn()
    out.zero_(), oute.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(oute, want[1])
    assert pkv.get_device_error() == 0


def test_calls_from_several_threads():
    servers = [Server(seed=50 + i) for i in range(4)]
    alone = [Server(seed=50 + i) for i in range(4)]
    torch.cuda.synchronize()

    def work(s, n=12):
        stream = torch.cuda.Stream()
        for _ in range(n):
            s.step(stream=stream)
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(s,)) for s in servers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for s in alone:
        work(s)
    for s, a in zip(servers, alone):
        assert torch.equal(s.out, a.out) and torch.equal(s.c.k, a.c.k) and torch.equal(s.c.vs, a.c.vs)
    assert pkv.get_device_error() == 0


def test_pools_beyond_32_bit_offsets():
    # 4.6 GB of codes per pool, 9 GB in a 16-bit one: blocks at the far end, through every call
    hq, hkv, d, bs = 8, 8, 128, 32
    nb = 280000
    k, v = (torch.zeros((nb, hkv, bs, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, hkv, bs, d // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    small = Mx4Case(BF16, hkv, d, bs, [100], seed=41)
    kn, vn, q = small.rows(100, hkv).cuda(), small.rows(100, hkv).cuda(), small.rows(100, hq).cuda()
    bt = torch.tensor([[nb - 1, nb - 7, 266000, 279000]], dtype=torch.int32, device="cuda")
    small.tables = np.arange(4, dtype=np.int32)[None]
    small.cuda()
    outs = []
    kept = ints(range(3, 99, 2))
    for kk, vv, s1, s2, t in ((k, v, ks, vs, bt), (small.k, small.v, small.ks, small.vs, small.bt)):
        pkv.kv_append_mx4(kk, vv, s1, s2, kn, vn, ints([0, 100]), ints([0]), t, 100)
        out, o2, o3 = torch.empty_like(q[:1]), torch.empty_like(q), torch.empty_like(q[:9])
        ws = torch.empty(pkv.decode_mx4_workspace_bytes(kk, 1, hq, 100, 0, 0, 2), dtype=torch.uint8, device="cuda")
        pkv.paged_decode_attn_mx4(kk, vv, s1, s2, q[:1], out, t, ints([100]), 0.1, 100, num_splits=2, workspace=ws)
        pkv.paged_extend_attn_mx4(kk, vv, s1, s2, q, o2, ints([0, 100]), ints([0]), t, 0.1, 100, 100)
        pkv.paged_extend_attn_mx4(kk, vv, s1, s2, q[:9], o3, ints([0, 9]), ints([91]), t, 0.1, 9, 100, window=40)
        p = pkv.KvPools([kk, vv, s1, s2])
        pkv.kv_compact(p, kept, ints([0, 48]), ints([1]), t, 48)
        far = ints([nb - 2 if kk is k else small.k.shape[0] - 1])
        pkv.kv_copy_blocks(p, t[0, :1].contiguous(), far)
        ko, vo, kc, vc = torch.empty_like(kn), torch.empty_like(vn), torch.empty_like(kn[:32]), torch.empty_like(vn[:32])
        pkv.kv_gather_mx4(kk, vv, s1, s2, ko, vo, ints([0, 100]), ints([0]), t)
        pkv.kv_gather_mx4(kk, vv, s1, s2, kc, vc, ints([0, 32]), ints([0]), far.view(1, 1))
        outs.append((out, o2, o3, ko, vo, kc, vc))
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert int(k[:260000].max()) == 0 and pkv.get_device_error() == 0
    del k, v
    pool = torch.zeros((140000, hkv, bs, d), dtype=torch.bfloat16, device="cuda")
    pool[139998].normal_()
    pkv.kv_copy_blocks(pkv.KvPools([pool]), ints([139998]), ints([139999]))
    assert torch.equal(pool[139999], pool[139998])
    pkv.kv_compact(pkv.KvPools([pool]), ints([5, 9, 40]), ints([0, 3]), ints([0]), ints([[139999, 139998]]), 3)
    assert torch.equal(pool[139999, :, :2], pool[139998, :, [5, 9]]) and torch.equal(pool[139999, :, 2], pool[139998, :, 8])
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("act", [F16, BF16])
def test_rows_off_a_32_byte_boundary(act):
    # rows that begin 16 bytes off: new rows, rows read back, queries and outputs
    hkv, d, bs, n = 3, 64, 16, 37
    c = Mx4Case(act, hkv, d, bs, [n], seed=3).cuda()

    def off(t):
        store = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        store[8:].copy_(t.flatten())
        return store[8:].view(t.shape)
    kn, vn = c.rows(n, hkv).cuda(), c.rows(n, hkv).cuda()
    a, b = Mx4Case(act, hkv, d, bs, [n], seed=3).cuda(), c
    pkv.kv_append_mx4(a.k, a.v, a.ks, a.vs, kn, vn, ints([0, n]), ints([0]), a.bt, n)
    pkv.kv_append_mx4(b.k, b.v, b.ks, b.vs, off(kn), off(vn), ints([0, n]), ints([0]), b.bt, n)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)
    ko, vo, ko2, vo2 = torch.empty_like(kn), torch.empty_like(vn), off(torch.zeros_like(kn)), off(torch.zeros_like(vn))
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko, vo, ints([0, n]), ints([0]), c.bt)
    pkv.kv_gather_mx4(c.k, c.v, c.ks, c.vs, ko2, vo2, ints([0, n]), ints([0]), c.bt)
    assert torch.equal(ko, ko2) and torch.equal(vo, vo2)
    q = c.rows(n, 6).cuda()
    out, out2 = torch.empty_like(q), off(torch.zeros_like(q))
    for x, o in ((q, out), (off(q), out2)):
        pkv.paged_extend_attn_mx4(c.k, c.v, c.ks, c.vs, x, o, ints([0, n]), ints([0]), c.bt, 0.1, n, n)
    assert torch.equal(out, out2) and pkv.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,bs,act", [(8, 2, 128, 16, BF16), (5, 1, 64, 32, F16), (2, 2, 64, 16, BF16),
                                             (12, 1, 128, 32, F16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_extend_of_few_rows(hq, hkv, d, bs, act, window, sinks):
    # requests whose rows fit one row tile, alone and many, over short and long prefixes
    for rows, prefix in (([1, 5, 0, 9], [300, 0, 17, 640]), ([10], [1500]), ([3] * 12, list(range(0, 480, 40)))):
        c = Mx4Case(act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=sum(rows)).cuda()
        q = c.rows(sum(rows), hq).cuda()
        out, lse = run_extend(c, q, hq, rows, prefix, window, sinks, False)
        check_attention(out, lse, extend_ref(c, q, hq, rows, prefix, window, sinks), act, d, f"{rows} {window}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("d,bs,act", [(64, 32, F16), (128, 16, BF16)])
def test_extend_of_more_items_than_sms(d, bs, act):
    # rows from none to many, several items per SM, read as codes and widened
    rows, prefix, hq = [0, 1100, 1, 0, 70, 2, 900], [9, 30, 40, 0, 200, 64, 0], 8
    c = Mx4Case(act, 8, d, bs, [p + n for p, n in zip(prefix, rows)], seed=12).cuda()
    q = c.rows(sum(rows), hq).cuda()
    ref = extend_ref(c, q, hq, rows, prefix)
    for work in (False, True):
        out, lse = run_extend(c, q, hq, rows, prefix, work=work)
        check_attention(out, lse, ref, act, d, f"{work}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("rows,prefix", [([16], [16]), ([20], [1500]), ([140], [0])])
def test_extend_scales_of_any_size(rows, prefix):
    # K's and V's scales 30 binary orders apart, beyond those that multiply in f16, and the least one
    c = Mx4Case(BF16, 2, 128, 16, [rows[0] + prefix[0]], seed=rows[0])
    c.vs = torch.from_numpy(c.rng.integers(100, 130, c.vs.shape).astype(np.uint8))
    c.ks = torch.from_numpy(c.rng.integers(95, 124, c.ks.shape).astype(np.uint8))
    blk = c.tables[0, 0]
    c.ks[blk], c.vs[blk] = 1, 1
    c.cuda()
    q = c.rows(rows[0], 8).cuda()
    vals = [to_f64(torch.from_numpy(x).float().half()) for x in c.values()]  # both take part as f16(code * scale)
    ref = R.attention(*vals, to_f64(q), [0, rows[0]], prefix, c.tables, 8, 1 / 128 ** 0.5)
    out, lse = run_extend(c, q, 8, rows, prefix, work=False)
    check_attention(out, lse, ref, BF16, 128)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("work", [False, True])
def test_extend_with_shared_blocks_nan_and_dirty_tail(work):
    # two requests read the same prefix blocks; scales behind the last token are NaN, then one that is seen
    rows, prefix = [25, 1100], [64, 64]
    c = Mx4Case(BF16, 2, 128, 16, [96, 1180], seed=12)
    c.tables[1, :4] = c.tables[0, :4]
    for b, n in enumerate((89, 1164)):
        blk = c.tables[b, n // 16]
        c.ks[blk, :, n % 16:], c.vs[blk, :, n % 16:] = 255, 255
    c.cuda()
    q = c.rows(sum(rows), 8).cuda()
    out, lse = run_extend(c, q, 8, rows, prefix, work=work)
    check_attention(out, lse, extend_ref(c, q, 8, rows, prefix), BF16, 128)
    c.vs[int(c.tables[0, 1]), 1, 3, 2] = 255   # V of a key that every row sees: dims 64 .. 95 of heads 4 .. 7
    bad, _ = run_extend(c, q, 8, rows, prefix, work=work)
    assert bool(torch.isnan(bad[:, 4:, 64:96]).all()) and torch.equal(bad[:, :4], out[:, :4])
    assert torch.equal(bad[:, 4:, :64], out[:, 4:, :64]) and torch.equal(bad[:, 4:, 96:], out[:, 4:, 96:])
    c.ks[int(c.tables[0, 1]), 0, 3, 2] = 255   # K: every row of heads 0 .. 3
    bad, lse = run_extend(c, q, 8, rows, prefix, work=work)
    assert bool(torch.isnan(bad[:, :4]).all()) and bool(torch.isnan(lse[:, :4]).all())
    assert pkv.get_device_error() == 0


def test_f16_values_beyond_the_range():
    # a code of 4 under a scale of 2^14 stands for 65536, more than f16 holds
    c = Mx4Case(F16, 1, 64, 16, [16], seed=13)
    c.v.fill_(0x66)
    c.vs.fill_(127 + 14)
    c.cuda()
    q = c.rows(16, 1).cuda()
    for work in (False, True):
        out, _ = run_extend(c, q, 1, [16], [0], work=work)
        assert bool((out == 65504.0).all())
    out, _ = run_decode(c, q[:1], 1, [16])                    # decode holds 65536 in fp32; f16 rounds it to inf
    assert bool(torch.isinf(out).all())


def test_nan_and_infinite_queries():
    c = Mx4Case(BF16, 1, 128, 16, [300, 300], seed=5).cuda()
    q = c.rows(2, 4).cuda()
    good, _ = run_decode(c, q, 4, [300, 300])
    q[0, 1, 7] = float("nan")
    for splits in (0, 1, 3):
        out, lse = run_decode(c, q, 4, [300, 300], splits=splits)
        assert bool(torch.isnan(out[0, 1]).all()) and bool(torch.isnan(lse[0, 1])) and bool(torch.isfinite(out[1]).all())
        assert bool(torch.isfinite(out[0, [0, 2, 3]]).all())
    out, _ = run_decode(c, q, 4, [300, 300])
    assert torch.equal(out[1], good[1])


def test_negative_and_zero_softmax_scales():
    c = Mx4Case(F16, 2, 64, 16, [90, 17], seed=6).cuda()
    q = c.rows(2, 4).cuda()
    for scale in (-0.2, 0.0, 3.0):
        out, lse = torch.empty_like(q), torch.empty((2, 4), device="cuda")
        pkv.paged_decode_attn_mx4(c.k, c.v, c.ks, c.vs, q, out, c.bt, ints([90, 17]), scale, 90, num_splits=1, lse_out=lse)
        ref = R.attention(*c.values(), to_f64(q), [0, 1, 2], [89, 16], c.tables, 4, scale)
        check_attention(out, lse, ref, F16, 64, f"{scale}")


def test_the_compiled_and_the_python_way():
    c = Mx4Case(BF16, 2, 64, 16, [40, 300], seed=3).cuda()
    kn, vn, q = c.rows(2, 2).cuda(), c.rows(2, 2).cuda(), c.rows(2, 8).cuda()
    direct, got = pkv._direct, []
    assert direct is not None
    try:
        for way in (direct, None):
            pkv._direct = way
            a = Mx4Case(BF16, 2, 64, 16, [40, 300], seed=3).cuda()
            out, oe, ko, vo = torch.empty_like(q), torch.empty_like(q), torch.empty_like(kn), torch.empty_like(vn)
            ws = torch.empty(pkv.decode_mx4_workspace_bytes(a.k, 2, 8, 300, 0, 0, 3), dtype=torch.uint8, device="cuda")
            pkv.kv_append_mx4(a.k, a.v, a.ks, a.vs, kn, vn, ints([0, 1, 2]), ints([39, 299]), a.bt, 1)
            pkv.paged_decode_attn_mx4(a.k, a.v, a.ks, a.vs, q, out, a.bt, ints([40, 300]), 0.1, 300, num_splits=3, workspace=ws)
            pkv.paged_extend_attn_mx4(a.k, a.v, a.ks, a.vs, q, oe, ints([0, 1, 2]), ints([39, 299]), a.bt, 0.1, 1, 300)
            p = pkv.KvPools([a.k, a.v, a.ks, a.vs])
            pkv.kv_copy_blocks(p, ints([0]), ints([1]))
            pkv.kv_compact(p, ints([8, 9]), ints([0, 2, 2]), ints([1, 0]), a.bt, 2)
            pkv.kv_gather_mx4(a.k, a.v, a.ks, a.vs, ko, vo, ints([0, 1, 2]), ints([1, 299]), a.bt)
            got.append([out, oe, ko, vo, a.k, a.v, a.ks, a.vs])
    finally:
        pkv._direct = direct
    assert all(torch.equal(x, y) for x, y in zip(*got)) and pkv.get_device_error() == 0
    with pytest.raises(ValueError, match="pool 1"):
        pkv.KvPools([c.k, c.ks[:3]])
    with pytest.raises(ValueError, match="contiguous"):
        pkv.KvPools([c.k, c.v[:, :1]])
    with pytest.raises(ValueError, match="device"):
        pkv.KvPools([c.k, c.v.cpu()])
    p = pkv.KvPools([c.k, c.v])
    with pytest.raises(ValueError, match="dst_blocks"):
        pkv.kv_copy_blocks(p, ints([1]), ints([1, 2]))
    with pytest.raises(ValueError, match="src_positions"):
        pkv.kv_compact(p, ints([1]).long(), ints([0, 1, 1]), ints([0, 0]), c.bt, 1)
    with pytest.raises(ValueError, match="device of the call"):
        pkv.kv_copy_blocks(p, torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(pkv.PkvError):
        pkv.kv_compact(pkv.KvPools([c.k, torch.zeros((c.k.shape[0], 2), device="cuda")]), ints([1]), ints([0, 1, 1]),
                       ints([0, 0]), c.bt, 1)

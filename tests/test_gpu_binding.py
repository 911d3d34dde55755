"""GPU checks of the compiled binding of the block-scaled, gather and window calls: the same results
and refusals as through the Python checks, and which arguments it leaves to them."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests.pkv_testlib import BF16
from tests.scaled_testlib import SCALED, Case, ints

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS, ROWS, PREFIX = 8, 2, 64, 16, [3, 40], [20, 5]
NAMES = ["append_block_scaled", "gather", "decode_window", "decode_block_scaled", "extend_window",
         "extend_block_scaled"]


class Calls:
    """The arguments of one call of each function, over one pair of pools."""

    def __init__(self):
        total = [p + n for p, n in zip(PREFIX, ROWS)]
        self.c = c = Case(SCALED, BF16, HKV, D, BS, total, seed=3).cuda()
        n = sum(ROWS)
        self.kn, self.vn, self.q = c.rows(n, HKV).cuda(), c.rows(n, HKV).cuda(), c.rows(n, HQ).cuda()
        self.qd = c.rows(2, HQ).cuda()
        self.ip, self.at, self.lens = ints([0, 3, 43]), ints(PREFIX), ints(total)
        self.ri, self.zero = ints([0, total[0], sum(total)]), ints([0, 0])
        need = pkv.decode_window_workspace_bytes(c.k, 2, HQ, 64, 0, 0, 3)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def args(self, name, **kw):
        """(function, positional, keyword arguments); kw replaces by name."""
        c, scale = self.c, D ** -0.5
        if name == "append_block_scaled":
            a = dict(k_cache=c.k, v_cache=c.v, k_scales=c.ks, v_scales=c.vs, k_new=self.kn, v_new=self.vn,
                     q_indptr=self.ip, prefix_lens=self.at, block_tables=c.bt, max_suffix_len=40)
            fn = pkv.kv_append_block_scaled
        elif name == "gather":
            ko = torch.full((sum(PREFIX) + sum(ROWS), HKV, D), 7.0, dtype=self.kn.dtype, device="cuda")
            a = dict(k_cache=c.k, v_cache=c.v, k_out=ko, v_out=ko.clone(), row_indptr=self.ri,
                     start_positions=self.zero, block_tables=c.bt, k_scales=c.ks, v_scales=c.vs)
            fn = pkv.kv_gather
        else:
            kind, form = name.split("_", 1)
            q = self.qd if kind == "decode" else self.q
            a = dict(k_cache=c.k, v_cache=c.v, q=q, out=torch.full_like(q, 7.0), block_tables=c.bt, sm_scale=scale, window=24,
                     sink_tokens=2, lse_out=torch.full((q.shape[0], HQ), 7.0, device="cuda"))
            if kind == "decode":
                a.update(seq_lens=self.lens, max_seq_len=64, num_splits=3, workspace=self.ws)
            else:
                a.update(q_indptr=self.ip, prefix_lens=self.at, max_suffix_len=40, max_total_len=64)
            a.update(dict(k_scales=c.ks, v_scales=c.vs) if form == "block_scaled" else dict(k_scale=0.5, v_scale=2.0))
            fn = getattr(pkv, f"paged_{kind}_attn_{form}")
        a.update(kw)
        return fn, a

    def run(self, name, **kw):
        fn, a = self.args(name, **kw)
        assert fn(**a) is None
        torch.cuda.synchronize()
        return [a[x] for x in ("k_cache", "v_cache", "k_scales", "v_scales", "k_out", "v_out", "out", "lse_out") if x in a]


class Spy:
    """Stands before the binding and counts the calls it took and the calls it left."""

    def __init__(self):
        self.took, self.left = 0, 0

    def __getattr__(self, name):
        assert name in NAMES
        fn = getattr(pkv._calls, name)

        def call(*a):
            st = fn(*a)
            self.took += st is not None
            self.left += st is None
            return st
        return call


@pytest.fixture(params=["compiled", "python"])
def way(request, monkeypatch):
    pkv.load()
    spy = Spy() if request.param == "compiled" else None
    monkeypatch.setattr(pkv, "_direct", spy)
    return spy


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("name", NAMES)
def test_the_same_results(name, monkeypatch):
    pkv.load()
    got = []
    for spy in (Spy(), None):
        monkeypatch.setattr(pkv, "_direct", spy)
        got.append([bits(t) for t in Calls().run(name)])
        assert spy is None or (spy.took, spy.left) == (1, 0)
    assert len(got[0]) == len(got[1]) and all(torch.equal(x, y) for x, y in zip(*got))
    assert pkv.get_device_error() == 0


class Sub(torch.Tensor):
    pass


@pytest.mark.parametrize("name", NAMES)
def test_arguments_of_other_kinds(name, monkeypatch):
    # what the Python functions convert keeps working, through them
    pkv.load()
    calls = Calls()
    monkeypatch.setattr(pkv, "_direct", None)
    want = [bits(t) for t in calls.run(name)]
    spy = Spy()
    monkeypatch.setattr(pkv, "_direct", spy)
    _, a = calls.args(name)
    kinds = [dict(block_tables=a["block_tables"].as_subclass(Sub))]
    if "window" in a:
        kinds += [dict(window=np.int32(24)), dict(window=24.0), dict(sm_scale=np.float64(a["sm_scale"]))]
    if name == "append_block_scaled":
        kinds += [dict(max_suffix_len=np.int64(40))]
    for kw in kinds:  # (appending the same rows again changes nothing)
        assert all(torch.equal(bits(t), w) for t, w in zip(calls.run(name, **kw), want)), kw
    assert (spy.took, spy.left) == (0, len(kinds))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert all(torch.equal(bits(t), w) for t, w in zip(calls.run(name, stream=side), want))
    with torch.cuda.stream(side):
        assert all(torch.equal(bits(t), w) for t, w in zip(calls.run(name), want))
    assert spy.took == 2 and pkv.get_device_error() == 0


@pytest.mark.parametrize("name", NAMES)
def test_refusals(name, way):
    calls = Calls()
    _, a = calls.args(name)
    tensors = {k: v for k, v in a.items() if isinstance(v, torch.Tensor)}
    before = {k: bits(v) for k, v in tensors.items()}
    bad = []
    for k, t in tensors.items():
        what = "cache" if k == "k_cache" else k
        if k != "k_cache":
            bad += [(ValueError, k, {k: t.cpu()})]
        if k == "workspace":
            bad += [(ValueError, k, {k: t[::2]})]
            continue
        bad += [(ValueError, what, {k: t[0]}),
                ((ValueError, TypeError), "", {k: t.double()}),
                (ValueError, "contiguous", {k: torch.stack([t, t], -1)[..., 0]})]
        if t.shape[0] > 1 and k not in ("k_cache", "q", "k_new", "k_out", "prefix_lens", "start_positions",
                                        "block_tables"):
            bad += [(ValueError, k, {k: t[:-1].clone()})]
    bad += [(pkv.PkvError, "", {"block_tables": a["block_tables"][:, :0].contiguous()})]
    if "window" in a:
        bad += [(pkv.PkvError, "", dict(sink_tokens=-1)), (pkv.PkvError, "", dict(sm_scale=float("nan")))]
    if "max_suffix_len" in a:
        bad += [(pkv.PkvError, "", dict(max_suffix_len=-1))]
    if name == "gather":
        bad += [(ValueError, "together", dict(k_scales=None)), (ValueError, "together", dict(v_scales=None)),
                (pkv.PkvError, "", dict(k_scale=0.0, k_scales=None, v_scales=None))]
    if name == "decode_block_scaled":
        bad += [(pkv.PkvError, "", dict(workspace=None)), (pkv.PkvError, "", dict(workspace=a["workspace"][:256]))]
    for kind, match, kw in bad:
        with pytest.raises(kind, match=match or None):
            calls.run(name, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(v), before[k]) for k, v in tensors.items()) and pkv.get_device_error() == 0


class Chain:
    """Calls that depend on one another and on small copies between them, without a pause: each is
    set up while the one before it still runs, and must not read before that has ended."""

    def __init__(self, steps=12):
        self.b = b = Calls()
        self.steps = steps
        gen = torch.Generator(device="cuda").manual_seed(5)
        draw = lambda t: torch.randn((steps,) + t.shape, generator=gen, device="cuda").to(t.dtype)
        self.kn, self.vn, self.q, self.qd = draw(b.kn), draw(b.vn), draw(b.q), draw(b.qd)
        self.extra = torch.randint(0, 9, (steps, 2), generator=gen, device="cuda", dtype=torch.int32)
        self.start = b.at.clone()
        self.got_q = torch.zeros((steps,) + b.q.shape, dtype=b.q.dtype, device="cuda")
        self.got_d = torch.zeros((steps,) + b.qd.shape, dtype=b.qd.dtype, device="cuda")
        self.got_k = torch.zeros((steps, 60, HKV, D), dtype=b.q.dtype, device="cuda")
        self.got_v = torch.zeros_like(self.got_k)
        self.rest = ints([0, 25, 60])

    def run(self, pause, side=None):
        b, c, main = self.b, self.b.c, torch.cuda.current_stream()
        for i in range(self.steps):
            for to, frm in ((b.kn, self.kn), (b.vn, self.vn), (b.q, self.q), (b.qd, self.qd)):
                to.copy_(frm[i])
            b.at.copy_(self.start).sub_(self.extra[i])
            b.lens.copy_(b.at)
            b.lens[0].add_(3)
            b.lens[1].add_(40)
            pause()
            pkv.kv_append_block_scaled(c.k, c.v, c.ks, c.vs, b.kn, b.vn, b.ip, b.at, c.bt, 40)
            pause()
            pkv.paged_extend_attn_block_scaled(c.k, c.v, c.ks, c.vs, b.q, self.got_q[i], b.ip, b.at, c.bt, 0.1, 40, 64)
            pause()
            if side is not None:  # the read back beside the decode
                side.wait_stream(main)
            with torch.cuda.stream(side or main):
                pkv.kv_gather(c.k, c.v, self.got_k[i], self.got_v[i], self.rest, b.zero, c.bt, k_scales=c.ks,
                              v_scales=c.vs)
            pause()
            for splits in (0, 3):
                pkv.paged_decode_attn_block_scaled(c.k, c.v, c.ks, c.vs, b.qd, self.got_d[i], c.bt, b.lens, 0.1, 64,
                                                   num_splits=splits, workspace=b.ws)
                pause()
                b.qd.copy_(self.got_d[i])
            pkv.paged_decode_attn_window(c.k, c.v, b.qd, self.got_d[i], c.bt, b.lens, 0.1, 64, 20, 3)
            pause()
            b.q.copy_(self.got_q[i])
            pkv.paged_extend_attn_window(c.k, c.v, b.q, self.got_q[i], b.ip, b.at, c.bt, 0.1, 40, 64, 20, 3)
            pause()
            if side is not None:
                main.wait_stream(side)
        return self

    def results(self):
        torch.cuda.synchronize()
        c = self.b.c
        return [bits(t) for t in (self.got_q, self.got_d, self.got_k, self.got_v, c.k, c.v, c.ks, c.vs)]


def test_calls_one_after_another_without_a_pause():
    want = Chain().run(torch.cuda.synchronize).results()
    assert not torch.equal(want[0][0], want[0][1])
    nothing = lambda: None
    for side in (None, torch.cuda.Stream()):
        for _ in range(3):
            assert all(torch.equal(x, y) for x, y in zip(Chain().run(nothing, side).results(), want))
    side = torch.cuda.Stream()
    for beside in (None, torch.cuda.Stream()):
        chain = Chain()
        before = [t.clone() for t in (chain.b.c.k, chain.b.c.v, chain.b.c.ks, chain.b.c.vs)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            chain.run(nothing, beside)
        for _ in range(3):
            for t, f in zip((chain.b.c.k, chain.b.c.v, chain.b.c.ks, chain.b.c.vs), before):
                t.copy_(f)
            graph.replay()
            assert all(torch.equal(x, y) for x, y in zip(chain.results(), want))
    # some of the drawn starts of the second request lie below 0: reported, its rows left alone
    assert bool((Chain().extra[:, 1] > PREFIX[1]).any()) and pkv.get_device_error() == 3


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_calls_wait_for_other_streams(name, captured):
    # an event of another stream between a call and the one before it in its stream: the inputs
    # arrive there late (a pause of about a millisecond, then the copies)
    pkv.load()
    calls, other, mine = Calls(), torch.cuda.Stream(), torch.cuda.Stream()
    _, a = calls.args(name)
    inputs = [a[k] for k in ("v_new" if "v_new" in a else "v_cache", "q", "k_new") if k in a]
    right = [t.clone() for t in inputs]
    kept = [t.clone() for t in (calls.c.k, calls.c.v, calls.c.ks, calls.c.vs)]
    want = [bits(t) for t in calls.run(name)]

    def restore():
        for t, f in zip((calls.c.k, calls.c.v, calls.c.ks, calls.c.vs), kept):
            t.copy_(f)
        for t in inputs:
            t.zero_()
        torch.cuda.synchronize()

    got = [t for t in (a.get(x) for x in ("k_cache", "v_cache", "k_scales", "v_scales", "k_out", "v_out", "out",
                                          "lse_out")) if t is not None]

    def work():  # on `mine`
        other.wait_stream(mine)
        with torch.cuda.stream(other):
            torch.cuda._sleep(2_000_000)
            for t, r in zip(inputs, right):
                t.copy_(r)
        before, b = calls.args("gather")
        before(**b)  # the call just before: its result is not looked at
        mine.wait_stream(other)
        calls.args(name)[0](**a)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=mine):
            work()
    for _ in range(3):
        restore()
        if captured:
            graph.replay()
        else:
            with torch.cuda.stream(mine):
                work()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(t), w) for t, w in zip(got, want))
    assert pkv.get_device_error() == 0


def test_calls_from_several_threads_at_once():
    pkv.load()
    # (the append first: appending the same rows again changes nothing)
    one = Calls()
    want = [[bits(t) for t in one.run(name)] for name in NAMES]
    failures = []

    def serve():
        try:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(stream):
                calls = Calls()
                for _ in range(30):
                    for name, w in zip(NAMES, want):
                        fn, a = calls.args(name)
                        fn(**a)
                        stream.synchronize()
                        got = [a[x] for x in ("k_cache", "v_cache", "k_scales", "v_scales", "k_out", "v_out", "out",
                                              "lse_out") if x in a]
                        assert all(torch.equal(bits(t), x) for t, x in zip(got, w)), name
        except BaseException as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=serve) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[0]
    assert pkv.get_device_error() == 0

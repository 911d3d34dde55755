"""Refusals of the microscaled and moving calls, without a GPU: the C ABI rejects bad arguments on the
host before it touches CUDA, and the binding checks tensors against one another."""
import ctypes

import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from paged_kv_cache_285_gb300 import build as pkv_build
from tests.test_abi import FAKE, _desc

ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


def mx4(**kw):
    return _desc(**{"cache_dtype": 3, "k_scale": 0.0, **kw})


def test_other_calls_refuse_the_dtype(lib):
    d = ctypes.byref(mx4(k_scale=1.0))
    assert lib.pkv_paged_decode_attn(d, FAKE, FAKE, FAKE, FAKE, 1, FAKE, 4, FAKE, 2, 4, 0.1, 64, 0, None, None, 0, None) == 1
    assert lib.pkv_kv_append(d, FAKE, FAKE, FAKE, FAKE, 1, FAKE, 4, None) == 1
    assert lib.pkv_kv_gather(d, FAKE, FAKE, None, None, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 4, 2, 5, None) == 1
    assert lib.pkv_paged_extend_attn(d, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 4, 1, 4, 0.1, 10, 10, 100, None, None, 0,
                                     None) == 1
    assert lib.pkv_kv_append_block_scaled(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 4, 2, 5, 3, None) == 1
    assert lib.pkv_decode_window_workspace_bytes(d, 2, 8, 1000, 0, 0, 4) == 0
    assert lib.pkv_extend_widen_workspace_bytes(d) == 0 and lib.pkv_extend_shared_prefix_workspace_bytes(d) == 0


def test_append_and_gather_refusals(lib):
    def append(desc=None, ks=FAKE, vs=FAKE, kn=FAKE, act=1, qi=FAKE, width=4, batch=2, rows=5, most=3, kc=FAKE):
        return lib.pkv_kv_append_mx4(ctypes.byref(desc or mx4()), kc, FAKE, ks, vs, kn, FAKE, act, qi, FAKE, FAKE, width,
                                     batch, rows, most, None)

    def gather(desc=None, ks=FAKE, ko=FAKE, act=1, ri=FAKE, width=4, batch=2, rows=5):
        return lib.pkv_kv_gather_mx4(ctypes.byref(desc or mx4()), FAKE, FAKE, ks, FAKE, ko, FAKE, act, ri, FAKE, FAKE, width,
                                     batch, rows, None)
    for call in (append, gather):
        assert call(desc=_desc()) == 2 and call(desc=_desc(cache_dtype=2)) == 2 and call(desc=mx4(cache_dtype=7)) == 1
        assert call(desc=mx4(head_dim=96)) == 2 and call(desc=mx4(block_size=64)) == 2 and call(desc=mx4(num_blocks=0)) == 1
        assert call(act=2) == 1 and call(act=3) == 1 and call(ks=None) == 1 and call(ks=ODD) == 1
        assert call(width=0) == 1 and call(batch=-1) == 1 and call(rows=-1) == 1
        assert call(batch=0) == 0 and call(rows=0) == 0
    assert append(kn=None) == 1 and append(kn=ODD) == 1 and append(qi=None) == 1 and append(most=-1) == 1
    assert append(vs=None) == 1 and append(kc=ODD) == 1 and append(most=0) == 0
    assert gather(ko=None) == 1 and gather(ko=ODD) == 1 and gather(ri=None) == 1


def test_attention_refusals(lib):
    def decode(desc=None, ks=FAKE, act=1, batch=2, hq=4, w=0, sinks=0, most=64, splits=0, q=FAKE, scale=0.1):
        return lib.pkv_paged_decode_attn_mx4(ctypes.byref(desc or mx4()), FAKE, FAKE, ks, FAKE, q, FAKE, act, FAKE, 4, FAKE,
                                             batch, hq, scale, most, w, sinks, splits, None, None, 0, None)

    def extend(desc=None, ks=FAKE, act=1, batch=2, hq=4, w=0, sinks=0, rows=20, ws=None, ws_bytes=0, scale=0.1):
        return lib.pkv_paged_extend_attn_mx4(ctypes.byref(desc or mx4()), FAKE, FAKE, ks, FAKE, FAKE, FAKE, act, FAKE, FAKE,
                                             FAKE, 4, batch, hq, scale, rows, 10, 100, w, sinks, None, ws, ws_bytes, None)
    for call in (decode, extend):
        assert call(desc=_desc()) == 2 and call(ks=None) == 1 and call(ks=ODD) == 1 and call(act=2) == 1
        assert call(w=-1) == 1 and call(sinks=-1) == 1 and call(hq=3) == 1 and call(batch=-1) == 1
        assert call(scale=float("nan")) == 1 and call(desc=mx4(head_dim=32)) == 2
        assert call(batch=0) == 0 and call(batch=0, ks=None) == 0
    assert decode(most=-1) == 1 and decode(q=None) == 1
    assert decode(most=10000, splits=2) in (3, 4)
    assert extend(rows=0) == 0 and extend(hq=2 * 129) == 2
    # the larger of the pools' 16-bit copies with their claims, and 152 parts of 256 rows (fp32, maximum and sum)
    need = lambda blocks: lib.pkv_extend_mx4_workspace_bytes(ctypes.byref(mx4(num_blocks=blocks)))  # noqa: E731
    assert need(8) == 152 * (256 * (128 * 4 + 8) + 32)
    assert need(8192) == 2 * 8192 * 2 * 16 * 128 * 2 + 256 * 257
    assert lib.pkv_extend_mx4_workspace_bytes(ctypes.byref(_desc())) == 0
    assert lib.pkv_decode_mx4_workspace_bytes(ctypes.byref(_desc()), 2, 8, 1000, 0, 0, 4) == 0
    f = lib.pkv_decode_mx4_workspace_bytes
    assert f(ctypes.byref(mx4()), 2, 8, 1000, 0, 50, 4) == lib.pkv_decode_workspace_bytes(ctypes.byref(_desc()), 2, 8, 1000, 4)
    assert f(ctypes.byref(mx4()), 2, 8, -1, 0, 0, 0) == 0


def pools(*rows):
    return (pkv.Pool * max(len(rows), 1))(*[pkv.Pool(*r) for r in rows])


GOOD = (0x10000, 8, 2, 16, 256)


def test_move_refusals(lib):
    def copy(ps, n=None, src=FAKE, pairs=3):
        return lib.pkv_kv_copy_blocks(ps, len(ps) if n is None else n, src, FAKE, pairs, None)

    def compact(ps, n=None, src=FAKE, width=4, batch=2, rows=5, most=3):
        return lib.pkv_kv_compact(ps, len(ps) if n is None else n, src, FAKE, FAKE, FAKE, width, batch, rows, most, None)
    for call in (copy, compact):
        assert call(pools(), 0) == 0 and call(pools(), -1) == 1 and call(None, 1) == 1
        assert call(pools((0, 8, 2, 16, 256))) == 1 and call(pools((0x10000, 0, 2, 16, 256))) == 1
        assert call(pools((0x10000, 8, 2, 16, 0))) == 1 and call(pools(GOOD, (0x10000, 9, 2, 16, 256))) == 1
        assert call(pools(GOOD), src=None) == 1
    assert copy(pools(GOOD), pairs=-1) == 1 and copy(pools(GOOD), pairs=0) == 0
    assert copy(pools((0x10002, 8, 2, 16, 256))) == 1 and copy(pools((0x10000, 8, 1, 1, 2))) == 1
    assert copy(pools((0x10000, 8, 1 << 16, 1 << 10, 256))) == 2
    assert compact(pools(GOOD), batch=-1) == 1 and compact(pools(GOOD), rows=-1) == 1 and compact(pools(GOOD), most=-1) == 1
    assert compact(pools(GOOD), width=0) == 1
    assert compact(pools(GOOD), batch=0) == 0 and compact(pools(GOOD), rows=0) == 0 and compact(pools(GOOD), most=0) == 0
    assert compact(pools(GOOD, (0x10000, 8, 3, 16, 256))) == 1 and compact(pools(GOOD, (0x10000, 8, 2, 32, 256))) == 1
    assert compact(pools((0x10000, 8, 2, 1, 4))) == 2           # a scale per block and head
    assert compact(pools((0x10000, 8, 2, 16, 48))) == 2 and compact(pools((0x10000, 8, 2, 16, 2048))) == 2
    assert compact(pools((0x10008, 8, 2, 16, 256))) == 1 and compact(pools((0x10001, 8, 2, 16, 2))) == 1


def test_binding_refusals(lib):
    c, s = torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 16, 4), dtype=torch.uint8)
    q, kn = torch.zeros((3, 8, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    bt, sl, ip = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    bad = [
        ("k_cache", lambda: pkv.kv_append_mx4(c.view(torch.int8), c, s, s, kn, kn, ip, sl, bt, 1)),
        ("v_cache", lambda: pkv.kv_append_mx4(c, c[:3], s, s, kn, kn, ip, sl, bt, 1)),
        ("k_scales", lambda: pkv.kv_append_mx4(c, c, s[..., :2], s, kn, kn, ip, sl, bt, 1)),
        ("v_scales", lambda: pkv.kv_append_mx4(c, c, s, s.float(), kn, kn, ip, sl, bt, 1)),
        ("k_new", lambda: pkv.kv_append_mx4(c, c, s, s, kn[..., :64], kn, ip, sl, bt, 1)),
        ("v_new", lambda: pkv.kv_append_mx4(c, c, s, s, kn, kn.half(), ip, sl, bt, 1)),
        ("q_indptr", lambda: pkv.kv_append_mx4(c, c, s, s, kn, kn, ip[:3], sl, bt, 1)),
        ("k_out", lambda: pkv.kv_gather_mx4(c, c, s, s, q, q, ip, sl, bt)),
        ("start_positions", lambda: pkv.kv_gather_mx4(c, c, s, s, kn, kn, ip, sl.long(), bt)),
        ("cache", lambda: pkv.paged_decode_attn_mx4(c[0], c, s, s, q, q.clone(), bt, sl, 0.1, 64)),
        ("seq_lens", lambda: pkv.paged_decode_attn_mx4(c, c, s, s, q, q.clone(), bt, sl[:2], 0.1, 64)),
        ("out", lambda: pkv.paged_extend_attn_mx4(c, c, s, s, q, q.half(), ip, sl, bt, 0.1, 8, 64)),
        ("device tensors", lambda: pkv.paged_decode_attn_mx4(c, c, s, s, q, q.clone(), bt, sl, 0.1, 64)),
        ("device tensors", lambda: pkv.kv_append_mx4(c, c, s, s, kn, kn, ip, sl, bt, 1)),
        ("device tensors", lambda: pkv.KvPools([c, s])),
        ("pool 0", lambda: pkv.KvPools([torch.zeros(4)])),
        ("KvPools", lambda: pkv.kv_copy_blocks([c], sl, sl)),
        ("KvPools", lambda: pkv.kv_compact([c], sl, ip, sl, bt, 1)),
        ("dst_blocks", lambda: pkv.kv_copy_blocks(pkv.KvPools([]), sl, sl[:2])),
        ("dst_starts", lambda: pkv.kv_compact(pkv.KvPools([]), sl, ip, sl.long(), bt, 1)),
        ("device tensors", lambda: pkv.kv_copy_blocks(pkv.KvPools([]), sl, sl)),
    ]
    for name, call in bad:
        with pytest.raises(ValueError, match=name):
            call()


def test_compiled_binding(lib):
    assert pkv._direct is not None
    t = torch.zeros(3)
    for name, n in [("append_mx4", 11), ("gather_mx4", 10), ("decode_mx4", 16), ("extend_mx4", 17), ("copy_blocks", 6),
                    ("compact", 9)]:
        fn = getattr(pkv._direct, name)
        c = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
        for args in ([t] * n, [None] * n, [c] * n, [c, c] + [1.0, 1.0] + [c] * (n - 4), [1 << 80] * n, [0, 0, -1] + [t] * (n - 3)):
            assert fn(*args) is None
        with pytest.raises(TypeError):
            fn(*([t] * (n - 1)))

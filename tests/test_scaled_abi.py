"""Refusals of the block-scaled and window calls, without a GPU: the C ABI rejects bad arguments on
the host before it touches CUDA, and the binding checks tensors against one another."""
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


def fp8(**kw):
    return _desc(cache_dtype=2, **kw)


def test_append_block_scaled_refusals(lib):
    def call(desc=None, ks=FAKE, vs=FAKE, kn=FAKE, act=1, qi=FAKE, width=4, batch=2, rows=5, most=3):
        return lib.pkv_kv_append_block_scaled(ctypes.byref(desc or fp8()), FAKE, FAKE, ks, vs, kn, FAKE, act, qi,
                                              FAKE, FAKE, width, batch, rows, most, None)
    assert call(desc=_desc()) == 2                      # a bf16 cache has no scales
    assert call(desc=_desc(cache_dtype=0), act=0) == 2
    assert call(desc=fp8(head_dim=96)) == 2 and call(desc=fp8(block_size=64)) == 2
    assert call(act=2) == 1                             # fp8 is not an act dtype
    assert call(ks=None) == 1 and call(vs=None) == 1 and call(ks=ctypes.c_void_p(0x10002)) == 1
    assert call(kn=None) == 1 and call(kn=ODD) == 1 and call(qi=None) == 1
    assert call(width=0) == 1 and call(batch=-1) == 1 and call(rows=-1) == 1 and call(most=-1) == 1
    assert call(batch=0) == 0 and call(rows=0) == 0 and call(most=0) == 0   # nothing to do
    assert lib.pkv_kv_append_block_scaled(None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 4, 2, 5,
                                          3, None) == 1


def test_gather_refusals(lib):
    def call(desc=None, ks=None, vs=None, ko=FAKE, act=1, ri=FAKE, width=4, batch=2, rows=5):
        return lib.pkv_kv_gather(ctypes.byref(desc or _desc()), FAKE, FAKE, ks, vs, ko, FAKE, act, ri, FAKE, FAKE,
                                 width, batch, rows, None)
    assert call(act=0) == 2                             # bf16 cache read as f16
    assert call(act=2) == 1
    assert call(ks=FAKE) == 1 and call(vs=FAKE) == 1    # one scale without the other
    assert call(ks=FAKE, vs=FAKE) == 2                  # a bf16 cache has no scales
    assert call(desc=fp8(), ks=ctypes.c_void_p(0x10002), vs=FAKE) == 1
    assert call(desc=fp8(k_scale=0.0)) == 1
    assert call(ko=None) == 1 and call(ko=ODD) == 1 and call(ri=None) == 1
    assert call(width=0) == 1 and call(batch=-1) == 1 and call(rows=-1) == 1
    assert call(batch=0) == 0 and call(rows=0) == 0


def test_decode_refusals(lib):
    def window(desc=None, act=1, batch=2, hq=4, w=32, sinks=4, most=64, splits=0, q=FAKE, scale=0.1):
        return lib.pkv_paged_decode_attn_window(ctypes.byref(desc or _desc()), FAKE, FAKE, q, FAKE, act, FAKE, 4,
                                                FAKE, batch, hq, scale, most, w, sinks, splits, None, None, 0, None)

    def scaled(desc=None, ks=FAKE, act=1, batch=2, hq=4, w=0, sinks=0, most=64, splits=0):
        return lib.pkv_paged_decode_attn_block_scaled(ctypes.byref(desc or fp8()), FAKE, FAKE, ks, FAKE, FAKE, FAKE,
                                                      act, FAKE, 4, FAKE, batch, hq, 0.1, most, w, sinks, splits,
                                                      None, None, 0, None)
    assert window(w=0) == 1 and window(w=-1) == 1 and window(sinks=-1) == 1
    assert window(hq=3) == 1 and window(act=0) == 2 and window(most=-1) == 1 and window(q=None) == 1
    assert window(scale=float("inf")) == 1 and window(desc=_desc(head_dim=32)) == 2
    assert window(batch=0) == 0
    assert scaled(desc=_desc()) == 2 and scaled(ks=None) == 1
    assert scaled(w=-1) == 1 and scaled(sinks=-1) == 1 and scaled(hq=3) == 1 and scaled(act=2) == 1
    assert scaled(batch=0) == 0 and scaled(batch=0, ks=None) == 0
    # two splits of a 300-token window need a workspace
    assert window(w=300, most=10000, splits=2) in (3, 4)


def test_extend_refusals(lib):
    def window(desc=None, w=32, sinks=0, hq=4, scale=0.1, rows=20, out=FAKE):
        return lib.pkv_paged_extend_attn_window(ctypes.byref(desc or _desc()), FAKE, FAKE, FAKE, out, 1, FAKE, FAKE,
                                                FAKE, 4, 2, hq, scale, rows, 10, 100, w, sinks, None, None, 0, None)

    def scaled(desc=None, ks=FAKE, w=0, sinks=0, ws=None, ws_bytes=0, batch=2):
        return lib.pkv_paged_extend_attn_block_scaled(ctypes.byref(desc or fp8()), FAKE, FAKE, ks, FAKE, FAKE, FAKE,
                                                      1, FAKE, FAKE, FAKE, 4, batch, 4, 0.1, 20, 10, 100, w, sinks,
                                                      None, ws, ws_bytes, None)
    assert window(w=0) == 1 and window(w=-5) == 1 and window(sinks=-1) == 1
    assert window(hq=3) == 1 and window(scale=-1.0) == 1 and window(hq=2 * 129) == 2 and window(out=ODD) == 1
    assert window(rows=0) == 0
    need = lib.pkv_extend_block_scaled_workspace_bytes(ctypes.byref(fp8()))
    assert need == 2 * 8 * 2 * 16 * 128 * 2 + 256       # two 16-bit pools and the claims
    assert lib.pkv_extend_block_scaled_workspace_bytes(ctypes.byref(_desc())) == 0
    assert scaled(desc=_desc()) == 2 and scaled(ks=None) == 1 and scaled(w=-1) == 1
    assert scaled(sinks=-1) == 1 and scaled(batch=-1) == 1 and scaled(batch=0) == 0


def test_decode_window_workspace_plan(lib):
    d = ctypes.byref(_desc())
    f = lib.pkv_decode_window_workspace_bytes
    # no window: the plain plan
    assert f(d, 2, 8, 1000, 0, 50, 4) == lib.pkv_decode_workspace_bytes(d, 2, 8, 1000, 4)
    # a window of 300 and 4 sinks: 19 + 1 + 1 tiles of 16 tokens, however long the sequence
    assert f(d, 2, 8, 1 << 30, 300, 4, 4) == lib.pkv_decode_workspace_bytes(d, 2, 8, 21 * 16, 4)
    # never more than the sequence itself
    assert f(d, 2, 8, 100, 1 << 30, 1 << 30, 4) == lib.pkv_decode_workspace_bytes(d, 2, 8, 100, 4)
    # a bound near 2^31 is planned as one a little below it
    for b in (1, 2, 64):
        assert 0 < f(d, b, 8, 2 ** 31 - 1, 0, 0, 0) == f(d, b, 8, 2 ** 31 - 2 ** 21 - 1, 0, 0, 0)
    assert f(d, 2, 8, -1, 3, 0, 0) == 0 and f(d, 2, 8, 10, -1, 0, 0) == 0 and f(d, 2, 8, 10, 1, -1, 0) == 0


def test_binding_refusals(lib):
    c = torch.zeros((4, 2, 16, 128), dtype=torch.uint8)
    c16 = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    s = torch.ones((4, 2))
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    kn = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    bt, sl, ip = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    bad = [
        ("k_scales", lambda: pkv.kv_append_block_scaled(c, c, s[:3], s, kn, kn, ip, sl, bt, 1)),
        ("v_scales", lambda: pkv.kv_append_block_scaled(c, c, s, s.double(), kn, kn, ip, sl, bt, 1)),
        ("v_new", lambda: pkv.kv_append_block_scaled(c, c, s, s, kn, kn.half(), ip, sl, bt, 1)),
        ("k_new", lambda: pkv.kv_append_block_scaled(c, c, s, s, q, q, ip, sl, bt, 1)),
        ("q_indptr", lambda: pkv.kv_append_block_scaled(c, c, s, s, kn, kn, ip[:3], sl, bt, 1)),
        ("prefix_lens", lambda: pkv.kv_append_block_scaled(c, c, s, s, kn, kn, ip, sl.long(), bt, 1)),
        ("block_tables", lambda: pkv.kv_append_block_scaled(c, c, s, s, kn, kn, ip, sl, bt[:2], 1)),
        ("together", lambda: pkv.kv_gather(c, c, kn, kn, ip, sl, bt, k_scales=s)),
        ("k_out", lambda: pkv.kv_gather(c, c, q, q, ip, sl, bt)),
        ("row_indptr", lambda: pkv.kv_gather(c, c, kn, kn, ip[:2], sl, bt)),
        ("k_scales", lambda: pkv.paged_decode_attn_block_scaled(c, c, s[:, :1], s, q, q.clone(), bt, sl, 0.1, 64)),
        ("seq_lens", lambda: pkv.paged_decode_attn_window(c16, c16, q, q.clone(), bt, sl[:2], 0.1, 64, 8)),
        ("lse_out", lambda: pkv.paged_extend_attn_window(c16, c16, q, q.clone(), ip, sl, bt, 0.1, 8, 64, 8,
                                                         lse_out=torch.zeros(3, 7))),
        ("v_scales", lambda: pkv.paged_extend_attn_block_scaled(c, c, s, s[:1], q, q.clone(), ip, sl, bt, 0.1, 8, 64)),
        ("device tensors", lambda: pkv.paged_decode_attn_window(c16, c16, q, q.clone(), bt, sl, 0.1, 64, 8)),
        ("device tensors", lambda: pkv.kv_append_block_scaled(c, c, s, s, kn, kn, ip, sl, bt, 1)),
    ]
    for name, call in bad:
        with pytest.raises(ValueError, match=name):
            call()


def test_compiled_binding(lib):
    # built for this torch and loaded; what is not on a device is left to the Python functions, which refuse it
    assert pkv._direct is not None and pkv._direct.torch_version == torch.__version__
    t = torch.zeros(3)
    for name, n in [("append_block_scaled", 11), ("gather", 12), ("decode_window", 16), ("decode_block_scaled", 16),
                    ("extend_window", 17), ("extend_block_scaled", 17)]:
        fn = getattr(pkv._direct, name)
        c = torch.zeros((4, 2, 16, 128), dtype=torch.uint8)
        for args in ([t] * n, [None] * n, [c] * n, [c, c] + [1.0, 1.0] + [c] * (n - 4), [1 << 80] * n):
            assert fn(*args) is None
        with pytest.raises(TypeError):
            fn(*([t] * (n - 1)))

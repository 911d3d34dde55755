"""Paged-KV attention for GB300 (sm_103a): a thin binding of libpkv.so (ctypes;
the calls that check their tensors in one pass through a compiled one, _calls.so).

Every call here only marshals arguments (PyTorch tensors -> device pointers,
the current CUDA stream) and forwards them to the C ABI declared in
``include/pkv.h``; all work runs in the library's CUDA kernels.  There is no
CPU fallback: if libpkv.so is missing or fails to load, every call raises.

The three calls (names as in pkv.h without the ``pkv_`` prefix):
  * kv_append          -- scatter new K/V rows into their cache slots;
  * paged_decode_attn  -- one query token per request over its paged K/V
                          (GQA, split-KV, online softmax, LSE merge);
  * paged_extend_attn  -- suffix prefill over cached prefix blocks + causal
                          suffix.
Also: paged_decode_attn_append and paged_extend_attn_append (the new tokens'
K/V written into the cache by the same call; in decode by the attention
kernel itself), paged_decode_attn_shared_prefix
(decode for groups of requests sharing a prefix, the prefix attended once per
group), RadixIndex (the host prefix index that hands out block tables and
prefix lengths; host int32 arrays in, host arrays out) and chain_hash (salted
chain hashes of full blocks, as block identifiers).

A cache of fp8 codes with a scale per block and kv head: kv_append_block_scaled
(quantised as it is written), paged_decode_attn_block_scaled and
paged_extend_attn_block_scaled; kv_gather reads rows back out of any cache.
paged_decode_attn_window and paged_extend_attn_window: attention with a
sliding window and a few first tokens that stay visible (the block-scaled calls
take a window too).

A cache of 4-bit floating-point codes with a scale per 32 values of a row:
kv_append_mx4, kv_gather_mx4, paged_decode_attn_mx4 and paged_extend_attn_mx4.
kv_copy_blocks and kv_compact move pages, and tokens within a request, in all
the pools of a KvPools.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
import warnings

import torch

__all__ = ["F16", "BF16", "FP8_E4M3", "PkvError", "CacheDesc", "lib_path", "load",
           "kv_append", "paged_decode_attn", "paged_extend_attn", "decode_workspace_bytes",
           "extend_workspace_bytes", "get_device_error", "status_string", "version",
           "paged_decode_attn_append", "RadixIndex", "NO_SPACE", "chain_hash",
           "paged_decode_attn_shared_prefix", "shared_prefix_decode_workspace_bytes",
           "paged_extend_attn_append", "paged_extend_attn_shared_prefix",
           "extend_shared_prefix_workspace_bytes", "extend_widen_workspace_bytes",
           "kv_append_block_scaled", "kv_gather", "decode_window_workspace_bytes",
           "paged_decode_attn_window", "paged_decode_attn_block_scaled",
           "paged_extend_attn_window", "extend_block_scaled_workspace_bytes",
           "paged_extend_attn_block_scaled", "MX4", "kv_append_mx4", "kv_gather_mx4",
           "decode_mx4_workspace_bytes", "paged_decode_attn_mx4", "extend_mx4_workspace_bytes",
           "extend_mx4_runs_workspace_bytes",
           "paged_extend_attn_mx4", "KvPools", "kv_copy_blocks", "kv_compact"]

F16, BF16, FP8_E4M3, MX4 = 0, 1, 2, 3
NO_SPACE = 5  # PKV_ERR_NO_SPACE
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpkv.so")
_lib = None
_direct = None  # _calls.so, the compiled binding of the small calls (set by load())
_lock = threading.Lock()


class RadixStats(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("free_blocks", ctypes.c_int32),
                ("tree_blocks", ctypes.c_int32), ("caller_blocks", ctypes.c_int32),
                ("nodes", ctypes.c_int32), ("evictable_leaves", ctypes.c_int32)]


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class CacheDesc(ctypes.Structure):
    """Mirror of pkv_cache_desc."""
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class Pool(ctypes.Structure):
    """Mirror of pkv_pool."""
    _fields_ = [("base", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("row_bytes", ctypes.c_int32)]


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libpkv.so (raises if it has not been built)."""
    global _lib, _direct
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run paged_kv_cache_285_gb300.build.build()")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        D = ctypes.POINTER(CacheDesc)
        lib.pkv_kv_append.argtypes = [D, P, P, P, P, ctypes.c_int, P, I32, P]
        lib.pkv_kv_append.restype = ctypes.c_int
        lib.pkv_decode_workspace_bytes.argtypes = [D, I32, I32, I32, I32]
        lib.pkv_decode_workspace_bytes.restype = SZ
        lib.pkv_paged_decode_attn.argtypes = [D, P, P, P, P, ctypes.c_int, P, I32, P, I32, I32, F,
                                              I32, I32, P, P, SZ, P]
        lib.pkv_paged_decode_attn.restype = ctypes.c_int
        lib.pkv_paged_decode_attn_append.argtypes = [D, P, P, P, P, P, P, ctypes.c_int, P, I32, P,
                                                      I32, I32, F, I32, I32, P, P, SZ, P]
        lib.pkv_paged_decode_attn_append.restype = ctypes.c_int
        lib.pkv_paged_decode_attn_noalloc.argtypes = [D, P, P, P, P, ctypes.c_int, P, I32, P, I32,
                                                       I32, F, I32, I32, P, P]
        lib.pkv_paged_decode_attn_noalloc.restype = ctypes.c_int
        lib.pkv_extend_workspace_bytes.argtypes = [D, I32, I32, I32, I32]
        lib.pkv_extend_workspace_bytes.restype = SZ
        lib.pkv_paged_extend_attn.argtypes = [D, P, P, P, P, ctypes.c_int, P, P, P, I32, I32, I32,
                                              F, I32, I32, I32, P, P, SZ, P]
        lib.pkv_paged_extend_attn.restype = ctypes.c_int
        lib.pkv_paged_extend_attn_append.argtypes = [D, P, P, P, P, P, P, ctypes.c_int, P, P, P, I32,
                                                     I32, I32, F, I32, I32, I32, P, P]
        lib.pkv_paged_extend_attn_append.restype = ctypes.c_int
        lib.pkv_paged_extend_attn_shared_prefix.argtypes = [D, P, P, P, P, ctypes.c_int, P, P, P,
                                                            I32, I32, I32, F, I32, P, P, I32, I32,
                                                            I32, P, P, SZ, P]
        lib.pkv_paged_extend_attn_shared_prefix.restype = ctypes.c_int
        lib.pkv_extend_shared_prefix_workspace_bytes.argtypes = [D]
        lib.pkv_extend_shared_prefix_workspace_bytes.restype = SZ
        lib.pkv_extend_widen_workspace_bytes.argtypes = [D]
        lib.pkv_extend_widen_workspace_bytes.restype = SZ
        lib.pkv_status_string.argtypes = [ctypes.c_int]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_get_device_error.argtypes = [ctypes.POINTER(I32), I32, P]
        lib.pkv_get_device_error.restype = ctypes.c_int
        lib.pkv_version.argtypes = []
        lib.pkv_version.restype = I32
        lib.pkv_shared_prefix_decode_workspace_bytes.argtypes = [D, I32, I32, I32, I32, I32]
        lib.pkv_shared_prefix_decode_workspace_bytes.restype = SZ
        lib.pkv_paged_decode_attn_shared_prefix.argtypes = [D, P, P, P, P, P, P, ctypes.c_int, P,
                                                             I32, P, I32, I32, F, P, P, I32, I32,
                                                             I32, I32, I32, P, P, SZ, P]
        lib.pkv_paged_decode_attn_shared_prefix.restype = ctypes.c_int
        lib.pkv_chain_hash.argtypes = [P, P, I32, I32, P, P, I32, P]
        lib.pkv_chain_hash.restype = ctypes.c_int
        I = ctypes.c_int
        lib.pkv_kv_append_block_scaled.argtypes = [D, P, P, P, P, P, P, I, P, P, P, I32, I32, I32,
                                                   I32, P]
        lib.pkv_kv_append_block_scaled.restype = I
        lib.pkv_kv_gather.argtypes = [D, P, P, P, P, P, P, I, P, P, P, I32, I32, I32, P]
        lib.pkv_kv_gather.restype = I
        lib.pkv_decode_window_workspace_bytes.argtypes = [D, I32, I32, I32, I32, I32, I32]
        lib.pkv_decode_window_workspace_bytes.restype = SZ
        lib.pkv_paged_decode_attn_window.argtypes = [D, P, P, P, P, I, P, I32, P, I32, I32, F, I32,
                                                     I32, I32, I32, P, P, SZ, P]
        lib.pkv_paged_decode_attn_window.restype = I
        lib.pkv_paged_decode_attn_block_scaled.argtypes = [D, P, P, P, P, P, P, I, P, I32, P, I32,
                                                           I32, F, I32, I32, I32, I32, P, P, SZ, P]
        lib.pkv_paged_decode_attn_block_scaled.restype = I
        lib.pkv_paged_extend_attn_window.argtypes = [D, P, P, P, P, I, P, P, P, I32, I32, I32, F,
                                                     I32, I32, I32, I32, I32, P, P, SZ, P]
        lib.pkv_paged_extend_attn_window.restype = I
        lib.pkv_extend_block_scaled_workspace_bytes.argtypes = [D]
        lib.pkv_extend_block_scaled_workspace_bytes.restype = SZ
        lib.pkv_paged_extend_attn_block_scaled.argtypes = [D, P, P, P, P, P, P, I, P, P, P, I32, I32,
                                                           I32, F, I32, I32, I32, I32, I32, P, P,
                                                           SZ, P]
        lib.pkv_paged_extend_attn_block_scaled.restype = I
        lib.pkv_kv_append_mx4.argtypes = [D, P, P, P, P, P, P, I, P, P, P, I32, I32, I32, I32, P]
        lib.pkv_kv_append_mx4.restype = I
        lib.pkv_kv_gather_mx4.argtypes = [D, P, P, P, P, P, P, I, P, P, P, I32, I32, I32, P]
        lib.pkv_kv_gather_mx4.restype = I
        lib.pkv_decode_mx4_workspace_bytes.argtypes = [D, I32, I32, I32, I32, I32, I32]
        lib.pkv_decode_mx4_workspace_bytes.restype = SZ
        lib.pkv_paged_decode_attn_mx4.argtypes = lib.pkv_paged_decode_attn_block_scaled.argtypes
        lib.pkv_paged_decode_attn_mx4.restype = I
        lib.pkv_extend_mx4_workspace_bytes.argtypes = [D]
        lib.pkv_extend_mx4_workspace_bytes.restype = SZ
        lib.pkv_extend_mx4_runs_workspace_bytes.argtypes = [D]
        lib.pkv_extend_mx4_runs_workspace_bytes.restype = SZ
        lib.pkv_paged_extend_attn_mx4.argtypes = lib.pkv_paged_extend_attn_block_scaled.argtypes
        lib.pkv_paged_extend_attn_mx4.restype = I
        lib.pkv_kv_copy_blocks.argtypes = [P, I32, P, P, I32, P]
        lib.pkv_kv_copy_blocks.restype = I
        lib.pkv_kv_compact.argtypes = [P, I32, P, P, P, P, I32, I32, I32, I32, P]
        lib.pkv_kv_compact.restype = I
        VP = ctypes.c_void_p
        lib.pkv_radix_create.argtypes = [I32, I32, ctypes.POINTER(VP)]
        lib.pkv_radix_create.restype = ctypes.c_int
        lib.pkv_radix_destroy.argtypes = [VP]
        lib.pkv_radix_destroy.restype = None
        lib.pkv_radix_match.argtypes = [VP, P, I32, P, I32, ctypes.POINTER(I32)]
        lib.pkv_radix_match.restype = ctypes.c_int
        lib.pkv_radix_release.argtypes = [VP, P, I32]
        lib.pkv_radix_release.restype = ctypes.c_int
        lib.pkv_radix_alloc.argtypes = [VP, I32, P]
        lib.pkv_radix_alloc.restype = ctypes.c_int
        lib.pkv_radix_free.argtypes = [VP, P, I32]
        lib.pkv_radix_free.restype = ctypes.c_int
        lib.pkv_radix_insert.argtypes = [VP, P, I32, P, P, ctypes.POINTER(I32)]
        lib.pkv_radix_insert.restype = ctypes.c_int
        lib.pkv_radix_evict.argtypes = [VP, I32, ctypes.POINTER(I32)]
        lib.pkv_radix_evict.restype = ctypes.c_int
        lib.pkv_radix_stats.argtypes = [VP, ctypes.POINTER(RadixStats)]
        lib.pkv_radix_stats.restype = ctypes.c_int
        # Tensors straight to the C ABI: without it (a build for another torch) the same calls
        # go through ctypes, 5 to 7 us more host time each.
        try:
            from . import _calls
            if _calls.torch_version != torch.__version__:
                raise ImportError(f"it is built for torch {_calls.torch_version}")
            _direct = _calls
        except ImportError as e:
            warnings.warn(f"_calls.so is not used ({e}): rebuild with build.build()")
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().pkv_status_string(int(status)).decode()


def version() -> int:
    return int(load().pkv_version())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.uint8 or t.dtype == getattr(torch, "float8_e4m3fn", None):
        return FP8_E4M3
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libpkv takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libpkv takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _desc(k_cache: torch.Tensor, k_scale: float, v_scale: float) -> CacheDesc:
    if k_cache.dim() != 4:
        raise ValueError("cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = k_cache.shape
    return CacheDesc(nb, bs, hkv, d, _dtype_code(k_cache), float(k_scale), float(v_scale))


def _need(dtype, **tensors):
    """The index tensors of a call must have the dtype the C ABI reads."""
    for name, t in tensors.items():
        if t is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _shape(name, t, shape, dtype=None):
    """A tensor argument must have the shape (and dtype) the call derives from the others: the
    C ABI takes bare pointers and cannot see how large a buffer is."""
    if t is None:
        return
    want = tuple(int(x) for x in shape)
    if tuple(t.shape) != want:
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _cache_pair(k_cache, v_cache):
    """K and V pools [num_blocks, num_kv_heads, block_size, head_dim] of one dtype; returns
    (num_kv_heads, head_dim)."""
    if k_cache.dim() != 4:
        raise ValueError("cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    _shape("v_cache", v_cache, k_cache.shape, k_cache.dtype)
    return int(k_cache.shape[1]), int(k_cache.shape[3])


def _rows(name, t, head_dim):
    """[rows, heads, head_dim] activations; returns (rows, heads)."""
    if t.dim() != 3 or int(t.shape[2]) != head_dim:
        raise ValueError(f"{name} must be [rows, heads, {head_dim}], got {tuple(t.shape)}")
    return int(t.shape[0]), int(t.shape[1])


def _table(name, t, rows):
    if t.dim() != 2 or int(t.shape[0]) != rows:
        raise ValueError(f"{name} must be [{rows}, max_blocks_per_seq], got {tuple(t.shape)}")


def _decode_shapes(k_cache, v_cache, q, out, block_tables, seq_lens, lse_out, k_new=None,
                   v_new=None):
    """Shapes of a decode call; returns (batch, num_q_heads)."""
    hkv, d = _cache_pair(k_cache, v_cache)
    b, hq = _rows("q", q, d)
    _shape("out", out, q.shape, q.dtype)
    _table("block_tables", block_tables, b)
    _shape("seq_lens", seq_lens, (b,))
    _shape("lse_out", lse_out, (b, hq), torch.float32)
    _shape("k_new", k_new, (b, hkv, d), q.dtype)
    _shape("v_new", v_new, (b, hkv, d), q.dtype)
    return b, hq


def _extend_shapes(k_cache, v_cache, q, out, q_indptr, prefix_lens, block_tables, lse_out,
                   k_new=None, v_new=None):
    """Shapes of an extend call; returns (total_q_rows, num_q_heads, batch)."""
    hkv, d = _cache_pair(k_cache, v_cache)
    rows, hq = _rows("q", q, d)
    _shape("out", out, q.shape, q.dtype)
    if prefix_lens.dim() != 1:
        raise ValueError("prefix_lens must be [batch]")
    batch = int(prefix_lens.shape[0])
    _shape("q_indptr", q_indptr, (batch + 1,))
    _table("block_tables", block_tables, batch)
    _shape("lse_out", lse_out, (rows, hq), torch.float32)
    _shape("k_new", k_new, (rows, hkv, d), q.dtype)
    _shape("v_new", v_new, (rows, hkv, d), q.dtype)
    return rows, hq, batch


def _check(status: int, what: str):
    if status != 0:
        raise PkvError(status, what)


def kv_append(k_cache, v_cache, k_new, v_new, slot_mapping, k_scale=1.0, v_scale=1.0,
              stream=None):
    """pkv_kv_append: k_new/v_new [T, Hkv, D] act dtype, slot_mapping int64 [T]."""
    _need(torch.int64, slot_mapping=slot_mapping)
    hkv, d = _cache_pair(k_cache, v_cache)
    if slot_mapping.dim() != 1:
        raise ValueError("slot_mapping must be [num_tokens]")
    t = int(slot_mapping.shape[0])
    _shape("k_new", k_new, (t, hkv, d))
    _shape("v_new", v_new, (t, hkv, d), k_new.dtype)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    st = lib.pkv_kv_append(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(k_new),
                           _ptr(v_new), _dtype_code(k_new), _ptr(slot_mapping),
                           int(slot_mapping.shape[0]), _stream(stream))
    _check(st, "pkv_kv_append")


def decode_workspace_bytes(k_cache, batch, num_q_heads, max_seq_len, num_splits=0,
                           k_scale=1.0, v_scale=1.0) -> int:
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    return int(lib.pkv_decode_workspace_bytes(ctypes.byref(desc), batch, num_q_heads,
                                              max_seq_len, num_splits))


def paged_decode_attn(k_cache, v_cache, q, out, block_tables, seq_lens, sm_scale, max_seq_len,
                      k_scale=1.0, v_scale=1.0, num_splits=0, lse_out=None, workspace=None,
                      stream=None):
    """pkv_paged_decode_attn: q/out [B, Hq, D]; block_tables int32 [B, W]; seq_lens int32 [B].
    ``workspace`` is a uint8 device tensor of at least decode_workspace_bytes() bytes."""
    _need(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
    b, hq = _decode_shapes(k_cache, v_cache, q, out, block_tables, seq_lens, lse_out)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.pkv_paged_decode_attn(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q),
                                   _ptr(out), _dtype_code(q), _ptr(block_tables),
                                   int(block_tables.shape[1]), _ptr(seq_lens), b, hq,
                                   float(sm_scale), int(max_seq_len), int(num_splits),
                                   _ptr(lse_out), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pkv_paged_decode_attn")


def paged_decode_attn_append(k_cache, v_cache, k_new, v_new, q, out, block_tables, seq_lens,
                             sm_scale, max_seq_len, k_scale=1.0, v_scale=1.0, num_splits=0,
                             lse_out=None, workspace=None, stream=None):
    """pkv_paged_decode_attn_append: k_new/v_new [B, Hkv, D] are written to position
    seq_len-1 of each request and attended in the same launch."""
    _need(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
    b, hq = _decode_shapes(k_cache, v_cache, q, out, block_tables, seq_lens, lse_out, k_new,
                           v_new)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.pkv_paged_decode_attn_append(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(out),
                                          _dtype_code(q), _ptr(block_tables),
                                          int(block_tables.shape[1]), _ptr(seq_lens), b, hq,
                                          float(sm_scale), int(max_seq_len), int(num_splits),
                                          _ptr(lse_out), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pkv_paged_decode_attn_append")


def paged_decode_attn_noalloc(k_cache, v_cache, q, out, block_tables, seq_lens, sm_scale,
                              max_seq_len, k_scale=1.0, v_scale=1.0, num_splits=0, lse_out=None,
                              stream=None):
    """pkv_paged_decode_attn_noalloc: paged_decode_attn with the split partials in the library's
    own scratch array (no workspace; calls on one device must not overlap)."""
    _need(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
    b, hq = _decode_shapes(k_cache, v_cache, q, out, block_tables, seq_lens, lse_out)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    st = lib.pkv_paged_decode_attn_noalloc(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache),
                                           _ptr(q), _ptr(out), _dtype_code(q), _ptr(block_tables),
                                           int(block_tables.shape[1]), _ptr(seq_lens), b, hq,
                                           float(sm_scale), int(max_seq_len), int(num_splits),
                                           _ptr(lse_out), _stream(stream))
    _check(st, "pkv_paged_decode_attn_noalloc")


def shared_prefix_decode_workspace_bytes(k_cache, batch, num_q_heads, max_prefix_len,
                                         max_suffix_len, num_splits=0) -> int:
    lib = load()
    desc = _desc(k_cache, 1.0, 1.0)
    return int(lib.pkv_shared_prefix_decode_workspace_bytes(ctypes.byref(desc), batch, num_q_heads,
                                                            max_prefix_len, max_suffix_len,
                                                            num_splits))


def paged_decode_attn_shared_prefix(k_cache, v_cache, q, out, block_tables, seq_lens, sm_scale,
                                    group_indptr, group_prefix_lens, max_group_size,
                                    max_prefix_len, max_suffix_len, k_new=None, v_new=None,
                                    num_splits=0, lse_out=None, workspace=None, stream=None,
                                    k_scale=1.0, v_scale=1.0):
    """pkv_paged_decode_attn_shared_prefix: requests [group_indptr[g], group_indptr[g+1])
    share their first group_prefix_lens[g] tokens (read through the group's first member's
    block table), attended once per group; max_prefix_len / max_suffix_len bound the groups'
    prefixes and the members' own tokens; k_new/v_new as paged_decode_attn_append; k_scale /
    v_scale are an fp8 cache's scales."""
    _need(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
    b, hq = _decode_shapes(k_cache, v_cache, q, out, block_tables, seq_lens, lse_out, k_new,
                           v_new)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    if group_indptr.dim() != 1:
        raise ValueError("group_indptr must be int32 [num_groups + 1]")
    ng = int(group_indptr.shape[0]) - 1
    if group_indptr.dtype != torch.int32 or group_prefix_lens.dtype != torch.int32:
        raise ValueError("group_indptr and group_prefix_lens must be int32")
    if tuple(group_prefix_lens.shape) != (ng,):
        raise ValueError("group_prefix_lens must be int32 [num_groups]")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.pkv_paged_decode_attn_shared_prefix(
        ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(q),
        _ptr(out), _dtype_code(q), _ptr(block_tables), int(block_tables.shape[1]), _ptr(seq_lens),
        b, hq, float(sm_scale), _ptr(group_indptr), _ptr(group_prefix_lens), ng,
        int(max_group_size), int(max_prefix_len), int(max_suffix_len), int(num_splits),
        _ptr(lse_out),
        _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pkv_paged_decode_attn_shared_prefix")


def extend_workspace_bytes(k_cache, batch, num_q_heads, total_q_rows, max_total_len,
                           k_scale=1.0, v_scale=1.0) -> int:
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    return int(lib.pkv_extend_workspace_bytes(ctypes.byref(desc), batch, num_q_heads,
                                              total_q_rows, max_total_len))


def paged_extend_attn(k_cache, v_cache, q, out, q_indptr, prefix_lens, block_tables, sm_scale,
                      max_suffix_len, max_total_len, k_scale=1.0, v_scale=1.0, lse_out=None,
                      workspace=None, stream=None):
    """pkv_paged_extend_attn: q/out [sum S, Hq, D]; q_indptr int32 [B+1]; prefix_lens int32 [B];
    workspace: None, or a uint8 device tensor of extend_widen_workspace_bytes() bytes or more
    (the pages read are then widened to 16 bits once per block; smaller ones are not used)."""
    _need(torch.int32, q_indptr=q_indptr, prefix_lens=prefix_lens, block_tables=block_tables)
    rows, hq, batch = _extend_shapes(k_cache, v_cache, q, out, q_indptr, prefix_lens,
                                     block_tables, lse_out)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.pkv_paged_extend_attn(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q),
                                   _ptr(out), _dtype_code(q), _ptr(q_indptr), _ptr(prefix_lens),
                                   _ptr(block_tables), int(block_tables.shape[1]), batch, hq,
                                   float(sm_scale), rows, int(max_suffix_len),
                                   int(max_total_len), _ptr(lse_out), _ptr(workspace), ws_bytes,
                                   _stream(stream))
    _check(st, "pkv_paged_extend_attn")


def extend_widen_workspace_bytes(k_cache, k_scale=1.0, v_scale=1.0) -> int:
    """pkv_extend_widen_workspace_bytes: the optional widening workspace of paged_extend_attn
    (16-bit copies of a bf16 cache's V pool or of an fp8 cache's K and V pools, and the
    per-block claims; 0 for an f16 cache)."""
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    return int(lib.pkv_extend_widen_workspace_bytes(ctypes.byref(desc)))


def extend_shared_prefix_workspace_bytes(k_cache, k_scale=1.0, v_scale=1.0) -> int:
    """pkv_extend_shared_prefix_workspace_bytes: the optional workspace of
    paged_extend_attn_shared_prefix (f16 copies of a bf16 cache's V pool or of an fp8
    cache's K and V pools; 0 for an f16 cache)."""
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    return int(lib.pkv_extend_shared_prefix_workspace_bytes(ctypes.byref(desc)))


def paged_extend_attn_shared_prefix(k_cache, v_cache, q, out, q_indptr, prefix_lens, block_tables,
                                    group_indptr, group_shared_lens, sm_scale, max_group_rows,
                                    max_total_len, k_scale=1.0, v_scale=1.0, lse_out=None,
                                    workspace=None, stream=None):
    """pkv_paged_extend_attn_shared_prefix: as paged_extend_attn, for groups of requests
    (group_indptr int32 [G+1], consecutive requests) sharing the blocks of their first
    group_shared_lens[g] tokens (int32 [G]); the groups' rows are packed into shared tiles.
    workspace: None, or a uint8 device tensor of extend_shared_prefix_workspace_bytes() bytes
    (the pages of a bf16 or fp8 cache are then widened to f16 once per call instead of per
    tile)."""
    _need(torch.int32, q_indptr=q_indptr, prefix_lens=prefix_lens, block_tables=block_tables,
          group_indptr=group_indptr, group_shared_lens=group_shared_lens)
    rows, hq, batch = _extend_shapes(k_cache, v_cache, q, out, q_indptr, prefix_lens,
                                     block_tables, lse_out)
    ng = int(group_indptr.shape[0]) - 1
    if group_indptr.dim() != 1 or ng < 0 or tuple(group_shared_lens.shape) != (ng,):
        raise ValueError("group_indptr must be [G+1] and group_shared_lens [G]")
    for name, t in (("group_indptr", group_indptr), ("group_shared_lens", group_shared_lens)):
        if t.device != q.device:
            raise ValueError(f"{name} must be on {q.device}")
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.pkv_paged_extend_attn_shared_prefix(
        ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q), _ptr(out), _dtype_code(q),
        _ptr(q_indptr), _ptr(prefix_lens), _ptr(block_tables), int(block_tables.shape[1]), batch,
        hq, float(sm_scale), rows, _ptr(group_indptr), _ptr(group_shared_lens), ng,
        int(max_group_rows), int(max_total_len), _ptr(lse_out), _ptr(workspace), ws_bytes,
        _stream(stream))
    _check(st, "pkv_paged_extend_attn_shared_prefix")


def paged_extend_attn_append(k_cache, v_cache, k_new, v_new, q, out, q_indptr, prefix_lens,
                             block_tables, sm_scale, max_suffix_len, max_total_len, lse_out=None,
                             stream=None, k_scale=1.0, v_scale=1.0):
    """pkv_paged_extend_attn_append: k_new/v_new [sum S, Hkv, D] (q's dtype) are written to
    positions prefix_lens[b] + i (an fp8 cache stores them quantised with k_scale / v_scale) and
    attended in the same call."""
    _need(torch.int32, q_indptr=q_indptr, prefix_lens=prefix_lens, block_tables=block_tables)
    rows, hq, batch = _extend_shapes(k_cache, v_cache, q, out, q_indptr, prefix_lens,
                                     block_tables, lse_out, k_new, v_new)
    lib = load()
    desc = _desc(k_cache, k_scale, v_scale)
    st = lib.pkv_paged_extend_attn_append(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(out),
                                          _dtype_code(q), _ptr(q_indptr), _ptr(prefix_lens),
                                          _ptr(block_tables), int(block_tables.shape[1]), batch,
                                          hq, float(sm_scale), rows, int(max_suffix_len),
                                          int(max_total_len), _ptr(lse_out), _stream(stream))
    _check(st, "pkv_paged_extend_attn_append")


# ---- calls over tensors of one device, checked in one pass (a decode step's host time is mostly
# these checks, so each tensor is looked at once and the C struct of a pool is kept by its values)

@functools.lru_cache(maxsize=256)
def _desc_ref(num_blocks, num_kv_heads, block_size, head_dim, code, k_scale, v_scale):
    return ctypes.byref(CacheDesc(num_blocks, block_size, num_kv_heads, head_dim, code, k_scale,
                                  v_scale))


def _refuse(name, t, shape, dtype, index):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index or not (t.is_cuda or index < 0):
        raise ValueError(f"{name} must be on the device of the call's other tensors, got {t.device}")
    raise ValueError(f"libpkv takes contiguous tensors: {name} is not")


def _arg(name, t, shape, dtype, index):
    """Data pointer of a tensor argument of this shape and dtype on the device of this index
    (-1: the CPU, refused by _run), contiguous."""
    if (t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != index or
            not t.is_contiguous()):
        _refuse(name, t, shape, dtype, index)
    return t.data_ptr()


def _workspace(t, index):
    """(pointer, bytes) of a workspace tensor of any shape and dtype, or of none."""
    if t is None:
        return None, 0
    if t.get_device() != index or not t.is_contiguous():
        _refuse("workspace", t, t.shape, t.dtype, index)
    return t.data_ptr(), t.numel() * t.element_size()


def _dim(name, t, dims, what):
    """The shape of a tensor of so many dimensions."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be {what}")
    return t.shape


_CODES = {torch.float16: F16, torch.bfloat16: BF16, torch.uint8: FP8_E4M3,
          getattr(torch, "float8_e4m3fn", torch.uint8): FP8_E4M3}


def _code(t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported tensor dtype {t.dtype}")
    return code


def _pools(k_cache, v_cache, k_scale, v_scale):
    """The desc of a pair of pools, their pointers, [num_blocks, Hkv], head dim, device index."""
    shape = _dim("cache", k_cache, 4, "[num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = shape
    dtype, index = k_cache.dtype, k_cache.get_device()
    return (_desc_ref(nb, hkv, bs, d, _code(k_cache), float(k_scale), float(v_scale)),
            _arg("k_cache", k_cache, shape, dtype, index),
            _arg("v_cache", v_cache, shape, dtype, index), (nb, hkv), d, index)


try:
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
except AttributeError:
    _current_device = torch.cuda.current_device

    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _run(what, index, stream, *args):
    """Call a C entry point whose last argument is the stream (None: the current one of device
    `index`), with that device current."""
    if index < 0:
        raise ValueError("libpkv takes device tensors")
    fn = getattr(_lib or load(), what)
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        st = fn(*args, s)
    else:
        with torch.cuda.device(index):
            st = fn(*args, s)
    if st != 0:
        raise PkvError(st, what)


def _layout(indptr_name, indptr, start_name, starts, block_tables, index):
    """Pointers of a call's row layout: indptr [B+1], starts [B], block_tables [B, W]; then B, W."""
    batch, = _dim(start_name, starts, 1, "[batch]")
    table = _dim("block_tables", block_tables, 2, "[batch, max_blocks_per_seq]")
    width = table[1]
    return (_arg(indptr_name, indptr, (batch + 1,), torch.int32, index),
            _arg(start_name, starts, (batch,), torch.int32, index),
            _arg("block_tables", block_tables, (batch, width), torch.int32, index), batch, width)


def kv_append_block_scaled(k_cache, v_cache, k_scales, v_scales, k_new, v_new, q_indptr,
                           prefix_lens, block_tables, max_suffix_len, stream=None):
    """pkv_kv_append_block_scaled: k_new/v_new [rows, Hkv, D] act dtype; row q_indptr[b] + i goes
    to position prefix_lens[b] + i of request b, quantised with a power-of-two scale per block
    and kv head.  k_scales/v_scales float32 [num_blocks, Hkv]; q_indptr int32 [B+1]; prefix_lens
    int32 [B]; max_suffix_len bounds the rows per request."""
    if _direct is not None:
        st = _direct.append_block_scaled(k_cache, v_cache, k_scales, v_scales, k_new, v_new,
                                         q_indptr, prefix_lens, block_tables, max_suffix_len,
                                         stream)
        if st is not None:
            return _check(st, "pkv_kv_append_block_scaled")
    desc, kc, vc, pages, d, dev = _pools(k_cache, v_cache, 1.0, 1.0)
    ks = _arg("k_scales", k_scales, pages, torch.float32, dev)
    vs = _arg("v_scales", v_scales, pages, torch.float32, dev)
    rows = _dim("k_new", k_new, 3, "[rows, num_kv_heads, head_dim]")[0]
    shape, dtype = (rows, pages[1], d), k_new.dtype
    kn = _arg("k_new", k_new, shape, dtype, dev)
    vn = _arg("v_new", v_new, shape, dtype, dev)
    qi, pl, bt, batch, width = _layout("q_indptr", q_indptr, "prefix_lens", prefix_lens,
                                       block_tables, dev)
    _run("pkv_kv_append_block_scaled", dev, stream, desc, kc, vc, ks, vs, kn, vn,
         _code(k_new), qi, pl, bt, width, batch, rows, int(max_suffix_len))


def kv_gather(k_cache, v_cache, k_out, v_out, row_indptr, start_positions, block_tables,
              k_scale=1.0, v_scale=1.0, k_scales=None, v_scales=None, stream=None):
    """pkv_kv_gather: rows row_indptr[b] .. row_indptr[b+1]-1 of k_out/v_out [rows, Hkv, D] (f16
    or bf16) are positions start_positions[b] ... of request b.  k_scale/v_scale: an fp8 cache's
    scales per tensor; k_scales/v_scales float32 [num_blocks, Hkv]: scales per block and head."""
    if _direct is not None:
        st = _direct.gather(k_cache, v_cache, k_out, v_out, row_indptr, start_positions,
                            block_tables, k_scale, v_scale, k_scales, v_scales, stream)
        if st is not None:
            return _check(st, "pkv_kv_gather")
    desc, kc, vc, pages, d, dev = _pools(k_cache, v_cache, k_scale, v_scale)
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales and v_scales come together")
    ks = vs = None
    if k_scales is not None:
        ks = _arg("k_scales", k_scales, pages, torch.float32, dev)
        vs = _arg("v_scales", v_scales, pages, torch.float32, dev)
    rows = _dim("k_out", k_out, 3, "[rows, num_kv_heads, head_dim]")[0]
    shape, dtype = (rows, pages[1], d), k_out.dtype
    ko = _arg("k_out", k_out, shape, dtype, dev)
    vo = _arg("v_out", v_out, shape, dtype, dev)
    ri, sp, bt, batch, width = _layout("row_indptr", row_indptr, "start_positions", start_positions,
                                       block_tables, dev)
    _run("pkv_kv_gather", dev, stream, desc, kc, vc, ks, vs, ko, vo, _code(k_out), ri, sp, bt,
         width, batch, rows)


def decode_window_workspace_bytes(k_cache, batch, num_q_heads, max_seq_len, window=0,
                                  sink_tokens=0, num_splits=0) -> int:
    """pkv_decode_window_workspace_bytes: the workspace of paged_decode_attn_window and
    paged_decode_attn_block_scaled; with num_splits 0 it serves every smaller batch and max_seq_len
    too."""
    desc = _desc(k_cache, 1.0, 1.0)
    return int(load().pkv_decode_window_workspace_bytes(ctypes.byref(desc), batch, num_q_heads,
                                                        max_seq_len, window, sink_tokens,
                                                        num_splits))


def _decode_args(q, out, block_tables, seq_lens, lse_out, head_dim, index):
    """Pointers of q, out, block_tables, seq_lens and lse_out, then batch, heads, table width."""
    b, hq, _ = _dim("q", q, 3, "[batch, num_q_heads, head_dim]")
    width = _dim("block_tables", block_tables, 2, "[batch, max_blocks_per_seq]")[1]
    shape, dtype = (b, hq, head_dim), q.dtype
    return (_arg("q", q, shape, dtype, index), _arg("out", out, shape, dtype, index),
            _arg("block_tables", block_tables, (b, width), torch.int32, index),
            _arg("seq_lens", seq_lens, (b,), torch.int32, index),
            None if lse_out is None else _arg("lse_out", lse_out, (b, hq), torch.float32, index),
            b, hq, width)


def paged_decode_attn_window(k_cache, v_cache, q, out, block_tables, seq_lens, sm_scale,
                             max_seq_len, window, sink_tokens=0, k_scale=1.0, v_scale=1.0,
                             num_splits=0, lse_out=None, workspace=None, stream=None):
    """pkv_paged_decode_attn_window: paged_decode_attn where each request's query sees its last
    `window` tokens and its first `sink_tokens`.  ``workspace`` is a uint8 device tensor of at
    least decode_window_workspace_bytes() bytes."""
    if _direct is not None:
        st = _direct.decode_window(k_cache, v_cache, k_scale, v_scale, q, out, block_tables,
                                   seq_lens, sm_scale, max_seq_len, window, sink_tokens, num_splits,
                                   lse_out, workspace, stream)
        if st is not None:
            return _check(st, "pkv_paged_decode_attn_window")
    desc, kc, vc, _, d, dev = _pools(k_cache, v_cache, k_scale, v_scale)
    qp, op, bt, sl, lse, b, hq, width = _decode_args(q, out, block_tables, seq_lens, lse_out, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _run("pkv_paged_decode_attn_window", dev, stream, desc, kc, vc, qp, op, _code(q), bt,
         width, sl, b, hq, float(sm_scale), int(max_seq_len), int(window), int(sink_tokens),
         int(num_splits), lse, ws, ws_bytes)


def paged_decode_attn_block_scaled(k_cache, v_cache, k_scales, v_scales, q, out, block_tables,
                                   seq_lens, sm_scale, max_seq_len, window=0, sink_tokens=0,
                                   num_splits=0, lse_out=None, workspace=None, stream=None):
    """pkv_paged_decode_attn_block_scaled: paged_decode_attn over fp8 codes with k_scales/v_scales
    float32 [num_blocks, Hkv]; window 0: every token, else as paged_decode_attn_window (the same
    workspace)."""
    if _direct is not None:
        st = _direct.decode_block_scaled(k_cache, v_cache, k_scales, v_scales, q, out, block_tables,
                                         seq_lens, sm_scale, max_seq_len, window, sink_tokens,
                                         num_splits, lse_out, workspace, stream)
        if st is not None:
            return _check(st, "pkv_paged_decode_attn_block_scaled")
    desc, kc, vc, pages, d, dev = _pools(k_cache, v_cache, 1.0, 1.0)
    ks = _arg("k_scales", k_scales, pages, torch.float32, dev)
    vs = _arg("v_scales", v_scales, pages, torch.float32, dev)
    qp, op, bt, sl, lse, b, hq, width = _decode_args(q, out, block_tables, seq_lens, lse_out, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _run("pkv_paged_decode_attn_block_scaled", dev, stream, desc, kc, vc, ks, vs, qp, op,
         _code(q), bt, width, sl, b, hq, float(sm_scale), int(max_seq_len), int(window),
         int(sink_tokens), int(num_splits), lse, ws, ws_bytes)


def _extend_args(q, out, q_indptr, prefix_lens, block_tables, lse_out, head_dim, index):
    """Pointers of q, out, the layout and lse_out, then rows, heads, batch, table width."""
    rows, hq, _ = _dim("q", q, 3, "[rows, num_q_heads, head_dim]")
    qi, pl, bt, batch, width = _layout("q_indptr", q_indptr, "prefix_lens", prefix_lens,
                                       block_tables, index)
    shape, dtype = (rows, hq, head_dim), q.dtype
    return (_arg("q", q, shape, dtype, index), _arg("out", out, shape, dtype, index), qi, pl, bt,
            None if lse_out is None else _arg("lse_out", lse_out, (rows, hq), torch.float32, index),
            rows, hq, batch, width)


def paged_extend_attn_window(k_cache, v_cache, q, out, q_indptr, prefix_lens, block_tables,
                             sm_scale, max_suffix_len, max_total_len, window, sink_tokens=0,
                             k_scale=1.0, v_scale=1.0, lse_out=None, workspace=None, stream=None):
    """pkv_paged_extend_attn_window: paged_extend_attn where the row at position p sees keys
    p - window + 1 .. p and the first `sink_tokens`.  workspace: optional, as there."""
    if _direct is not None:
        st = _direct.extend_window(k_cache, v_cache, k_scale, v_scale, q, out, q_indptr,
                                   prefix_lens, block_tables, sm_scale, max_suffix_len,
                                   max_total_len, window, sink_tokens, lse_out, workspace, stream)
        if st is not None:
            return _check(st, "pkv_paged_extend_attn_window")
    desc, kc, vc, _, d, dev = _pools(k_cache, v_cache, k_scale, v_scale)
    qp, op, qi, pl, bt, lse, rows, hq, batch, width = _extend_args(
        q, out, q_indptr, prefix_lens, block_tables, lse_out, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _run("pkv_paged_extend_attn_window", dev, stream, desc, kc, vc, qp, op, _code(q), qi, pl,
         bt, width, batch, hq, float(sm_scale), rows, int(max_suffix_len), int(max_total_len),
         int(window), int(sink_tokens), lse, ws, ws_bytes)


def extend_block_scaled_workspace_bytes(k_cache) -> int:
    """pkv_extend_block_scaled_workspace_bytes: the optional workspace of
    paged_extend_attn_block_scaled (16-bit copies of the K and V pools, and the per-block
    claims)."""
    desc = _desc(k_cache, 1.0, 1.0)
    return int(load().pkv_extend_block_scaled_workspace_bytes(ctypes.byref(desc)))


def paged_extend_attn_block_scaled(k_cache, v_cache, k_scales, v_scales, q, out, q_indptr,
                                   prefix_lens, block_tables, sm_scale, max_suffix_len,
                                   max_total_len, window=0, sink_tokens=0, lse_out=None,
                                   workspace=None, stream=None):
    """pkv_paged_extend_attn_block_scaled: paged_extend_attn over fp8 codes with k_scales/v_scales
    float32 [num_blocks, Hkv]; window 0: every key, else as paged_extend_attn_window.
    workspace: None, or a uint8 device tensor of extend_block_scaled_workspace_bytes() bytes or
    more (calls with many rows per request then widen the pages they read once per block)."""
    if _direct is not None:
        st = _direct.extend_block_scaled(k_cache, v_cache, k_scales, v_scales, q, out, q_indptr,
                                         prefix_lens, block_tables, sm_scale, max_suffix_len,
                                         max_total_len, window, sink_tokens, lse_out, workspace,
                                         stream)
        if st is not None:
            return _check(st, "pkv_paged_extend_attn_block_scaled")
    desc, kc, vc, pages, d, dev = _pools(k_cache, v_cache, 1.0, 1.0)
    ks = _arg("k_scales", k_scales, pages, torch.float32, dev)
    vs = _arg("v_scales", v_scales, pages, torch.float32, dev)
    qp, op, qi, pl, bt, lse, rows, hq, batch, width = _extend_args(
        q, out, q_indptr, prefix_lens, block_tables, lse_out, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _run("pkv_paged_extend_attn_block_scaled", dev, stream, desc, kc, vc, ks, vs, qp, op,
         _code(q), qi, pl, bt, width, batch, hq, float(sm_scale), rows,
         int(max_suffix_len), int(max_total_len), int(window), int(sink_tokens), lse, ws, ws_bytes)


def _pools_mx4(k_cache, v_cache, k_scales, v_scales):
    """The desc of pools of e2m1 codes, the pointers of pools and scales, Hkv, head dim, device."""
    shape = _dim("cache", k_cache, 4, "[num_blocks, num_kv_heads, block_size, head_dim / 2]")
    nb, hkv, bs, half = shape
    index = k_cache.get_device()
    scales = (nb, hkv, bs, half // 16)
    return (_desc_ref(nb, hkv, bs, 2 * half, MX4, 1.0, 1.0),
            _arg("k_cache", k_cache, shape, torch.uint8, index),
            _arg("v_cache", v_cache, shape, torch.uint8, index),
            _arg("k_scales", k_scales, scales, torch.uint8, index),
            _arg("v_scales", v_scales, scales, torch.uint8, index), hkv, 2 * half, index)


def _desc_mx4(k_cache):
    nb, hkv, bs, half = _dim("cache", k_cache, 4, "[num_blocks, num_kv_heads, block_size, head_dim / 2]")
    return _desc_ref(nb, hkv, bs, 2 * half, MX4, 1.0, 1.0)


def kv_append_mx4(k_cache, v_cache, k_scales, v_scales, k_new, v_new, q_indptr, prefix_lens,
                  block_tables, max_suffix_len, stream=None):
    """pkv_kv_append_mx4: k_new/v_new [rows, Hkv, D] act dtype; row q_indptr[b] + i goes to position
    prefix_lens[b] + i of request b, quantised to e2m1 codes (k_cache/v_cache uint8
    [num_blocks, Hkv, block_size, D / 2]) with a power-of-two scale per 32 values
    (k_scales/v_scales uint8 [num_blocks, Hkv, block_size, D / 32]).  q_indptr int32 [B+1];
    prefix_lens int32 [B]; max_suffix_len bounds the rows per request."""
    if _direct is not None:
        st = _direct.append_mx4(k_cache, v_cache, k_scales, v_scales, k_new, v_new, q_indptr,
                                prefix_lens, block_tables, max_suffix_len, stream)
        if st is not None:
            return _check(st, "pkv_kv_append_mx4")
    desc, kc, vc, ks, vs, hkv, d, dev = _pools_mx4(k_cache, v_cache, k_scales, v_scales)
    rows = _dim("k_new", k_new, 3, "[rows, num_kv_heads, head_dim]")[0]
    shape, dtype = (rows, hkv, d), k_new.dtype
    kn = _arg("k_new", k_new, shape, dtype, dev)
    vn = _arg("v_new", v_new, shape, dtype, dev)
    qi, pl, bt, batch, width = _layout("q_indptr", q_indptr, "prefix_lens", prefix_lens,
                                       block_tables, dev)
    _run("pkv_kv_append_mx4", dev, stream, desc, kc, vc, ks, vs, kn, vn, _code(k_new), qi, pl, bt,
         width, batch, rows, int(max_suffix_len))


def kv_gather_mx4(k_cache, v_cache, k_scales, v_scales, k_out, v_out, row_indptr, start_positions,
                  block_tables, stream=None):
    """pkv_kv_gather_mx4: rows row_indptr[b] .. row_indptr[b+1]-1 of k_out/v_out [rows, Hkv, D] (f16
    or bf16) are positions start_positions[b] ... of request b of a cache that kv_append_mx4
    wrote."""
    if _direct is not None:
        st = _direct.gather_mx4(k_cache, v_cache, k_scales, v_scales, k_out, v_out, row_indptr,
                                start_positions, block_tables, stream)
        if st is not None:
            return _check(st, "pkv_kv_gather_mx4")
    desc, kc, vc, ks, vs, hkv, d, dev = _pools_mx4(k_cache, v_cache, k_scales, v_scales)
    rows = _dim("k_out", k_out, 3, "[rows, num_kv_heads, head_dim]")[0]
    shape, dtype = (rows, hkv, d), k_out.dtype
    ko = _arg("k_out", k_out, shape, dtype, dev)
    vo = _arg("v_out", v_out, shape, dtype, dev)
    ri, sp, bt, batch, width = _layout("row_indptr", row_indptr, "start_positions", start_positions,
                                       block_tables, dev)
    _run("pkv_kv_gather_mx4", dev, stream, desc, kc, vc, ks, vs, ko, vo, _code(k_out), ri, sp, bt,
         width, batch, rows)


def decode_mx4_workspace_bytes(k_cache, batch, num_q_heads, max_seq_len, window=0, sink_tokens=0,
                               num_splits=0) -> int:
    """pkv_decode_mx4_workspace_bytes: the workspace of paged_decode_attn_mx4; with num_splits 0 it
    serves every smaller batch and max_seq_len too."""
    return int(load().pkv_decode_mx4_workspace_bytes(_desc_mx4(k_cache), batch, num_q_heads,
                                                     max_seq_len, window, sink_tokens, num_splits))


def paged_decode_attn_mx4(k_cache, v_cache, k_scales, v_scales, q, out, block_tables, seq_lens,
                          sm_scale, max_seq_len, window=0, sink_tokens=0, num_splits=0, lse_out=None,
                          workspace=None, stream=None):
    """pkv_paged_decode_attn_mx4: paged_decode_attn over e2m1 codes with microscales (the pools of
    kv_append_mx4); window 0: every token, else as paged_decode_attn_window.  ``workspace`` is a
    uint8 device tensor of at least decode_mx4_workspace_bytes() bytes."""
    if _direct is not None:
        st = _direct.decode_mx4(k_cache, v_cache, k_scales, v_scales, q, out, block_tables, seq_lens,
                                sm_scale, max_seq_len, window, sink_tokens, num_splits, lse_out,
                                workspace, stream)
        if st is not None:
            return _check(st, "pkv_paged_decode_attn_mx4")
    desc, kc, vc, ks, vs, _, d, dev = _pools_mx4(k_cache, v_cache, k_scales, v_scales)
    qp, op, bt, sl, lse, b, hq, width = _decode_args(q, out, block_tables, seq_lens, lse_out, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _run("pkv_paged_decode_attn_mx4", dev, stream, desc, kc, vc, ks, vs, qp, op, _code(q), bt, width,
         sl, b, hq, float(sm_scale), int(max_seq_len), int(window), int(sink_tokens),
         int(num_splits), lse, ws, ws_bytes)


def extend_mx4_workspace_bytes(k_cache) -> int:
    """pkv_extend_mx4_workspace_bytes: the optional workspace of paged_extend_attn_mx4 (16-bit copies
    of the K and V pools and the per-block claims, or the parts of calls that are shared out)."""
    return int(load().pkv_extend_mx4_workspace_bytes(_desc_mx4(k_cache)))


def extend_mx4_runs_workspace_bytes(k_cache) -> int:
    """pkv_extend_mx4_runs_workspace_bytes: the part of it that calls with few rows over long prefixes
    use, which does not grow with the pools."""
    return int(load().pkv_extend_mx4_runs_workspace_bytes(_desc_mx4(k_cache)))


def paged_extend_attn_mx4(k_cache, v_cache, k_scales, v_scales, q, out, q_indptr, prefix_lens,
                          block_tables, sm_scale, max_suffix_len, max_total_len, window=0,
                          sink_tokens=0, lse_out=None, workspace=None, stream=None):
    """pkv_paged_extend_attn_mx4: paged_extend_attn over e2m1 codes with microscales; window 0: every
    key, else as paged_extend_attn_window.  workspace: None, or a uint8 device tensor of
    extend_mx4_workspace_bytes() bytes or more (calls with many rows per request then widen the pages
    they read once per block, calls with few rows over long prefixes are shared out over all SMs), or of
    extend_mx4_runs_workspace_bytes() (the latter alone)."""
    if _direct is not None:
        st = _direct.extend_mx4(k_cache, v_cache, k_scales, v_scales, q, out, q_indptr, prefix_lens,
                                block_tables, sm_scale, max_suffix_len, max_total_len, window,
                                sink_tokens, lse_out, workspace, stream)
        if st is not None:
            return _check(st, "pkv_paged_extend_attn_mx4")
    desc, kc, vc, ks, vs, _, d, dev = _pools_mx4(k_cache, v_cache, k_scales, v_scales)
    qp, op, qi, pl, bt, lse, rows, hq, batch, width = _extend_args(
        q, out, q_indptr, prefix_lens, block_tables, lse_out, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _run("pkv_paged_extend_attn_mx4", dev, stream, desc, kc, vc, ks, vs, qp, op, _code(q), qi, pl, bt,
         width, batch, hq, float(sm_scale), rows, int(max_suffix_len), int(max_total_len),
         int(window), int(sink_tokens), lse, ws, ws_bytes)


class KvPools:
    """The pools that kv_copy_blocks and kv_compact move pages and tokens in: K, V and scales of any
    layers, contiguous device tensors [num_blocks, num_kv_heads, block_size, ...] of any dtypes, or
    [num_blocks, num_kv_heads] (a scale per block and kv head: copied, not compacted).  They are
    checked once, here, and held for as long as this object."""

    def __init__(self, pools):
        self.tensors = tuple(pools)
        self._count, self._index = len(self.tensors), -1
        if _direct is not None:
            got = _direct.pools(self.tensors)
            if got is not None:
                self._array, self._at, self._index = got
                return
        rows = []
        for i, t in enumerate(self.tensors):
            if not isinstance(t, torch.Tensor) or t.dim() < 2:
                raise ValueError(f"pool {i} must be a tensor [num_blocks, num_kv_heads, ...]")
            index = t.get_device()
            if not t.is_cuda or (i > 0 and index != self._index):
                raise ValueError(f"libpkv takes device tensors of one device: pool {i} is on {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"libpkv takes contiguous tensors: pool {i} is not")
            shape, size = t.shape, t.element_size()
            nb, hkv = shape[0], shape[1]
            bs = shape[2] if len(shape) > 2 else 1
            for n in shape[3:]:
                size *= n
            if i > 0 and nb != rows[0][1]:
                raise ValueError(f"pool {i} must have {rows[0][1]} blocks, got {tuple(shape)}")
            if not 0 < min(nb, hkv, bs, size) <= max(nb, hkv, bs, size) <= 2 ** 31 - 1:
                raise ValueError(f"pool {i} is empty or too large: {tuple(shape)}")
            rows.append((t.data_ptr(), nb, hkv, bs, size))
            self._index = index
        order = sorted(range(self._count), key=lambda i: rows[i][0])
        for i, j in zip(order, order[1:]):
            if rows[i][0] + rows[i][1] * rows[i][2] * rows[i][3] * rows[i][4] > rows[j][0]:
                raise ValueError(f"pools {i} and {j} overlap")
        self._array = (Pool * self._count)(*rows)
        self._at = ctypes.addressof(self._array)


def kv_copy_blocks(pools, src_blocks, dst_blocks, stream=None):
    """pkv_kv_copy_blocks: block dst_blocks[i] becomes what src_blocks[i] holds in every pool of a
    KvPools; int32 [pairs] each, a pair with a negative id is skipped."""
    if _direct is not None and type(pools) is KvPools:
        st = _direct.copy_blocks(pools._at, pools._count, pools._index, src_blocks, dst_blocks, stream)
        if st is not None:
            return _check(st, "pkv_kv_copy_blocks")
    if not isinstance(pools, KvPools):
        raise ValueError("pools must be a KvPools")
    pairs, = _dim("src_blocks", src_blocks, 1, "[pairs]")
    dev = src_blocks.get_device() if pools._count == 0 else pools._index
    src = _arg("src_blocks", src_blocks, (pairs,), torch.int32, dev)
    dst = _arg("dst_blocks", dst_blocks, (pairs,), torch.int32, dev)
    _run("pkv_kv_copy_blocks", dev, stream, pools._at, pools._count, src, dst, pairs)


def kv_compact(pools, src_positions, row_indptr, dst_starts, block_tables, max_rows, stream=None):
    """pkv_kv_compact: in every pool of a KvPools the token at position
    src_positions[row_indptr[b] + i] of request b goes to position dst_starts[b] + i, in place, as
    if all were read first.  src_positions int32 [rows], rising within a request; row_indptr int32
    [B+1]; dst_starts int32 [B]; max_rows bounds the rows per request."""
    if _direct is not None and type(pools) is KvPools:
        st = _direct.compact(pools._at, pools._count, pools._index, src_positions, row_indptr,
                             dst_starts, block_tables, max_rows, stream)
        if st is not None:
            return _check(st, "pkv_kv_compact")
    if not isinstance(pools, KvPools):
        raise ValueError("pools must be a KvPools")
    rows, = _dim("src_positions", src_positions, 1, "[rows]")
    dev = src_positions.get_device() if pools._count == 0 else pools._index
    src = _arg("src_positions", src_positions, (rows,), torch.int32, dev)
    ri, ds, bt, batch, width = _layout("row_indptr", row_indptr, "dst_starts", dst_starts, block_tables,
                                       dev)
    _run("pkv_kv_compact", dev, stream, pools._at, pools._count, src, ri, ds, bt, width, batch, rows,
         int(max_rows))


def chain_hash(tokens, token_indptr, block_size, hashes, salts=None, stream=None):
    """pkv_chain_hash: tokens int32 [T], token_indptr int32 [B+1], hashes int64 [B, max_blocks]
    (uint64 bits), salts int64 [B] (uint64 bits) or None; all device tensors."""
    lib = load()
    b = int(token_indptr.shape[0]) - 1
    if tokens.dtype != torch.int32 or token_indptr.dtype != torch.int32 or token_indptr.dim() != 1:
        raise ValueError("tokens and token_indptr must be int32 (token_indptr 1-D)")
    if hashes.dtype != torch.int64 or hashes.dim() != 2 or hashes.shape[0] != b:
        raise ValueError("hashes must be int64 [batch, max_blocks]")
    if salts is not None and (salts.dtype != torch.int64 or tuple(salts.shape) != (b,)):
        raise ValueError("salts must be int64 [batch]")
    _check(lib.pkv_chain_hash(_ptr(tokens), _ptr(token_indptr), b, int(block_size), _ptr(salts),
                              _ptr(hashes), int(hashes.shape[1]), _stream(stream)), "pkv_chain_hash")


def get_device_error(clear=True, stream=None) -> int:
    """Read (and by default clear) the library's device error word (synchronises)."""
    lib = load()
    w = ctypes.c_int32(0)
    _check(lib.pkv_get_device_error(ctypes.byref(w), int(bool(clear)), _stream(stream)),
           "pkv_get_device_error")
    return int(w.value)


def _host_i32(a):
    """Contiguous host int32 array and its address (numpy or a CPU tensor)."""
    import numpy as np
    if isinstance(a, torch.Tensor):
        a = a.detach().to("cpu").numpy()
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return arr, (arr.ctypes.data if arr.size else None)


class RadixIndex:
    """pkv_radix_*: host prefix index over the block ids [0, num_blocks) of one pool.
    Token and block lists are host int32 arrays; results are numpy int32 arrays."""

    def __init__(self, block_size: int, num_blocks: int):
        self._lib = load()
        h = ctypes.c_void_p()
        _check(self._lib.pkv_radix_create(int(block_size), int(num_blocks), ctypes.byref(h)),
               "pkv_radix_create")
        self._h = h
        self.block_size = int(block_size)

    def close(self):
        if getattr(self, "_h", None):
            self._lib.pkv_radix_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def match(self, tokens):
        """(matched_tokens, blocks): the locked longest cached whole-block prefix."""
        import numpy as np
        t, tp = _host_i32(tokens)
        cap = t.size // self.block_size
        out = np.zeros(max(cap, 1), dtype=np.int32)
        m = ctypes.c_int32(0)
        _check(self._lib.pkv_radix_match(self._h, tp, int(t.size), out.ctypes.data, cap, ctypes.byref(m)),
               "pkv_radix_match")
        return int(m.value), out[: m.value // self.block_size].copy()

    def release(self, tokens, matched_tokens: int):
        t, tp = _host_i32(tokens)
        _check(self._lib.pkv_radix_release(self._h, tp, int(matched_tokens)), "pkv_radix_release")

    def alloc(self, count: int):
        import numpy as np
        out = np.zeros(max(int(count), 1), dtype=np.int32)
        _check(self._lib.pkv_radix_alloc(self._h, int(count), out.ctypes.data), "pkv_radix_alloc")
        return out[: int(count)].copy()

    def free(self, blocks):
        b, bp = _host_i32(blocks)
        _check(self._lib.pkv_radix_free(self._h, bp, int(b.size)), "pkv_radix_free")

    def insert(self, tokens, blocks):
        """Adopt the full blocks of a request; returns the caller blocks that were freed
        because the tree already held the same tokens."""
        import numpy as np
        t, tp = _host_i32(tokens)
        b, bp = _host_i32(blocks)
        rel = np.zeros(max(t.size // self.block_size, 1), dtype=np.int32)
        n = ctypes.c_int32(0)
        _check(self._lib.pkv_radix_insert(self._h, tp, int(t.size), bp, rel.ctypes.data, ctypes.byref(n)),
               "pkv_radix_insert")
        return rel[: n.value].copy()

    def evict(self, num_blocks: int) -> int:
        f = ctypes.c_int32(0)
        _check(self._lib.pkv_radix_evict(self._h, int(num_blocks), ctypes.byref(f)), "pkv_radix_evict")
        return int(f.value)

    def stats(self) -> dict:
        st = RadixStats()
        _check(self._lib.pkv_radix_stats(self._h, ctypes.byref(st)), "pkv_radix_stats")
        return {k: int(getattr(st, k)) for k, _ in RadixStats._fields_}

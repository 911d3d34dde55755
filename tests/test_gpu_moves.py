"""GPU checks of kv_copy_blocks and kv_compact: whole pools of every kind, bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from oracle import mx4_ref as M
from tests.scaled_testlib import ints

pytestmark = pytest.mark.gpu


def pools_of(kinds, nb, hkv, bs, d, seed):
    """Random pools; kinds: f16, bf16, fp8, mx4 (codes), mx (their scales), scale (one per block and head)."""
    rng = np.random.default_rng(seed)
    shape = {"f16": (bs, 2 * d), "bf16": (bs, 2 * d), "fp8": (bs, d), "mx4": (bs, d // 2), "mx": (bs, d // 32), "scale": (4,)}
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "scale": torch.float32, "fp8": torch.float8_e4m3fn}
    got = []
    for kind in kinds:
        x = torch.from_numpy(rng.integers(0, 256, (nb, hkv) + shape[kind]).astype(np.uint8)).cuda()
        x = x.view(dtype.get(kind, torch.uint8))
        got.append(x.view(nb, hkv) if kind == "scale" else x)
    return got


def raw(t):
    """The bytes of a pool [num_blocks, hkv, ...] on the host."""
    return t.contiguous().view(torch.uint8).cpu().numpy()


ALL = ["bf16", "mx4", "scale", "mx", "fp8", "f16"]


@pytest.mark.parametrize("kinds,hkv,bs,d", [(["bf16"], 1, 16, 64), (ALL, 3, 16, 128), (ALL, 8, 32, 64), (ALL * 25, 2, 16, 64),
                                            (["scale"], 1, 16, 64), (["f16", "f16"], 8, 32, 128)])
def test_copy_blocks(kinds, hkv, bs, d):
    nb = 40
    pools = pools_of(kinds, nb, hkv, bs, d, seed=hkv + d)
    perm = np.random.default_rng(4).permutation(nb)
    src = [int(x) for x in perm[[0, 1, 2, 1, 1, 3]]] + [-1, 5, int(perm[30])]
    dst = [int(x) for x in perm[[10, 11, 12, 13, 14, 15]]] + [7, -3, int(perm[30])]
    before = [raw(t) for t in pools]
    pkv.kv_copy_blocks(pkv.KvPools(pools), ints(src), ints(dst))
    assert pkv.get_device_error() == 0
    for t, want in zip(pools, before):
        want = want.copy()
        old = want.copy()
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                want[b] = old[a]
        np.testing.assert_array_equal(raw(t), want)


def test_copy_blocks_of_pools_in_the_middle_of_a_tensor():
    # pools that begin 4 and 16 bytes off a 32-byte boundary, and one of odd size
    store = torch.randint(0, 1 << 30, (4096,), dtype=torch.int32, device="cuda")
    for off, row in ((1, 8), (4, 16), (0, 5), (8, 24)):
        pool = store[off:off + 10 * 2 * row].view(10, 2, row)
        before = raw(store.view(1, -1))[0]
        pkv.kv_copy_blocks(pkv.KvPools([pool]), ints([3, 3]), ints([9, 0]))
        want = before.copy()
        size = 2 * row * 4
        for b in (9, 0):
            want[4 * off + b * size:4 * off + (b + 1) * size] = before[4 * off + 3 * size:4 * off + 4 * size]
        np.testing.assert_array_equal(raw(store.view(1, -1))[0], want)


def test_pools_that_overlap_are_refused():
    t = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    for pools in ([t, t], [t[4:], t[2:6]], [t[2:6], t[:4], t[4:]]):
        with pytest.raises(ValueError, match="overlap"):
            pkv.KvPools(pools)
    pkv.KvPools([t[4:], t[:4]])


def test_pools_read_by_the_compiled_and_the_python_way():
    class Named(torch.Tensor):
        pass

    pools = pools_of(ALL, 9, 3, 32, 64, seed=1) + [torch.zeros((9, 3), device="cuda").as_subclass(Named)]
    direct, got = pkv._direct, []
    assert direct is not None and direct.pools(tuple(pools)) is None and direct.pools(tuple(pools[:6])) is not None
    try:
        for way in (direct, None):
            pkv._direct = way
            p = pkv.KvPools(pools[:6])
            got.append((bytes(p._array), p._count, p._index))
        assert got[0] == got[1] and pkv.KvPools([])._count == 0
    finally:
        pkv._direct = direct
    assert pkv.KvPools(pools)._count == 7
    for bad in (pools[:1] + [pools[1][:5]], pools[:1] + [pools[1].cpu()], pools[:1] + [None], [pools[1][:, :2]], [pools[1][:0]]):
        assert direct.pools(tuple(bad)) is None
        with pytest.raises((ValueError, TypeError)):
            pkv.KvPools(bad)


def test_copy_blocks_reports():
    pools = pools_of(["bf16", "mx"], 12, 2, 16, 64, seed=1)
    before = [raw(t) for t in pools]
    p = pkv.KvPools(pools)
    pkv.kv_copy_blocks(p, ints([12, 1]), ints([3, 12]))
    assert pkv.get_device_error() == 1
    pkv.kv_copy_blocks(p, ints([]), ints([]))
    pkv.kv_copy_blocks(p, ints([2 ** 31 - 1]), ints([0]))
    assert pkv.get_device_error() == 1
    for t, want in zip(pools, before):
        np.testing.assert_array_equal(raw(t), want)
    # beside a bad pair the others are copied
    pkv.kv_copy_blocks(p, ints([12, 1]), ints([3, 4]))
    assert pkv.get_device_error() == 1 and bool(torch.equal(pools[0][4].view(torch.uint8), pools[0][1].view(torch.uint8)))


def moves(rng, starts, counts, spread):
    src, ip = [], [0]
    for s, n in zip(starts, counts):
        src += sorted(int(x) for x in s + rng.choice(max(1, int(n * spread)), n, replace=False)) if n else []
        ip.append(len(src))
    return src, ip


TOKENS = ["bf16", "mx4", "mx", "fp8", "f16"]
COMPACTS = [
    # kinds, hkv, bs, d, starts, counts, spread
    (["bf16"], 1, 16, 64, [0], [1], 9),
    (TOKENS, 3, 16, 128, [5, 0, 33, 16], [7, 0, 40, 130], 2.2),
    (TOKENS, 2, 32, 64, [0, 17], [300, 5], 3),
    (["bf16", "bf16"], 8, 16, 128, [300, 20, 7], [5, 1, 6], 4),   # accepted drafts
    (["f16", "mx"], 1, 16, 128, [2], [5000], 1.3),                # few, long: clusters, many passes
    (["fp8"], 2, 32, 128, [0], [3000], 1.9),
    (["mx"], 12, 16, 64, [1, 1, 1], [900, 3, 70], 1.5),
    (TOKENS * 27, 2, 16, 64, [3, 9], [20, 33], 2),                # more pools than a launch takes
    (["bf16", "mx"], 40, 16, 128, [3], [50], 2),                  # two heads a CTA
    (["bf16"] * 4, 150, 16, 128, [3, 0], [9, 1], 2),              # 14 heads a CTA, the last one fewer
    (["bf16"] * 12, 8, 16, 128, [0, 9, 3, 0, 1], [40, 900, 0, 500, 700], 1.5),  # rounds of CTAs, the longest first
    (["bf16"] * 4, 8, 16, 64, [0] * 32, [70, 20] * 15 + [300, 300], 1.5),
    (["fp8"] * 4, 8, 32, 128, [0, 1, 2] * 11, [300] + [70, 1] * 16, 1.5),       # ... and more requests than are ranked
]


@pytest.mark.parametrize("cfg", COMPACTS, ids=lambda c: f"{len(c[0])}{c[0][0]}-h{c[1]}-bs{c[2]}-d{c[3]}-n{max(c[5])}")
def test_compact(cfg):
    kinds, hkv, bs, d, starts, counts, spread = cfg
    rng = np.random.default_rng(sum(counts))
    src, ip = moves(rng, starts, counts, spread)
    ends = [max(src[ip[b]:ip[b + 1]] + [s + n]) + 1 for b, (s, n) in enumerate(zip(starts, counts))]
    need = [-(-e // bs) for e in ends]
    nb = sum(need) + 2
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(starts), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    pools = pools_of(kinds, nb, hkv, bs, d, seed=d)
    before = [raw(t) for t in pools]
    pkv.kv_compact(pkv.KvPools(pools), ints(src), ints(ip), ints(starts), torch.from_numpy(tables).cuda(), max(max(counts), 1))
    assert pkv.get_device_error() == 0
    for t, old in zip(pools, before):
        np.testing.assert_array_equal(raw(t), M.compact(old, src, ip, starts, tables))


def test_compact_again_and_again():
    # the same moves time after time, each on what the one before left
    pools = pools_of(["fp8", "mx"], 70, 2, 16, 128, seed=2)
    rng = np.random.default_rng(2)
    src, ip = moves(rng, [7], [500], 2)
    tables = rng.permutation(70)[None].astype(np.int32)
    p, bt = pkv.KvPools(pools), torch.from_numpy(tables).cuda()
    want = [raw(t) for t in pools]
    for _ in range(6):
        pkv.kv_compact(p, ints(src), ints(ip), ints([7]), bt, 500)
        want = [M.compact(w, src, ip, [7], tables) for w in want]
    for t, w in zip(pools, want):
        np.testing.assert_array_equal(raw(t), w)


def test_compact_reports():
    pools = pools_of(["bf16"], 12, 2, 16, 64, seed=1)
    p, bt = pkv.KvPools(pools), torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    before = raw(pools[0])
    call = lambda src, ip, to, most, t=bt: pkv.kv_compact(p, ints(src), ints(ip), ints(to), t, most)  # noqa: E731

    def untouched(code):
        assert pkv.get_device_error() == code
        np.testing.assert_array_equal(raw(pools[0]), before)

    call([], [0, 0, 0], [0, 0], 0)
    untouched(0)
    call([9], [0, 0, 1], [-1, -1], 1)                   # a negative destination
    untouched(3)
    call([9, 10], [0, 3, 3], [0, 0], 3)                 # rows that the call does not have
    untouched(3)
    call([96], [0, 1, 1], [0, 0], 1)                    # past the table
    untouched(3)
    call([3], [0, 1, 1], [4, 0], 1)                     # before its destination
    untouched(3)
    bad = bt.clone()
    bad[0, 1], bad[1, 0] = -1, 12
    call([17], [0, 1, 1], [0, 0], 1, bad)
    untouched(1)
    call([40], [0, 0, 1], [0, 0], 1, bad)
    untouched(1)
    call([5, 5], [0, 2, 2], [0, 0], 2)                  # not rising: the second is not moved
    want = before.copy()
    want[0, :, 0] = before[0, :, 5]
    assert pkv.get_device_error() == 3
    np.testing.assert_array_equal(raw(pools[0]), want)
    call([20, 30], [0, 2, 2], [0, 0], 1)                # beyond the hint
    want[0, :, 0] = before[1, :, 4]
    assert pkv.get_device_error() == 3
    np.testing.assert_array_equal(raw(pools[0]), want)

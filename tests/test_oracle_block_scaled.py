"""Pins of the float64 references of the block-scaled cache and of windowed attention (no GPU)."""
import numpy as np
import torch

from oracle import block_scaled_ref as R
from oracle import ref_numpy


def test_codes_against_pytorch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.decode(codes), want, equal_nan=True)
    finite = codes[np.isfinite(want)]
    assert np.array_equal(R.encode(R.decode(finite)), finite)
    mid = (R._VALUES[1:] + R._VALUES[:-1]) / 2  # every tie
    x = np.concatenate([mid, -mid, np.random.default_rng(0).uniform(-448, 448, 5000)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x), want)
    assert list(R.encode([1e9, -1e9, np.inf, -np.inf, np.nan, 449.0])) == [0x7E, 0xFE, 0x7E, 0xFE, 0x7F, 0x7E]


def test_scale_by_hand():
    s = lambda *v: R.scale_of(np.array(v))  # noqa: E731
    assert s(448.0) == 1.0 and s(448.1) == 2.0 and s(224.0) == 0.5 and s(-1.0, 0.5) == 2.0 ** -8
    assert s(0.0) == R.MIN_SCALE and s(np.inf, np.nan, 7.0) == 2.0 ** -6
    assert s(np.inf) == R.MIN_SCALE and s(3.3e38) == 2.0 ** 120


def test_append_keeps_and_grows():
    codes, scales = np.zeros((3, 1, 16, 2), np.uint8), np.full((3, 1), 7.0, np.float32)
    t = [[2, 0]]
    one = np.array([[[448.0, -1.0]]])
    c, s = R.append(codes, scales, one, [0, 1], [0], t)
    assert s[2, 0] == 1.0 and list(R.decode(c[2, 0, 0])) == [448.0, -1.0] and np.array_equal(s[:2], scales[:2])
    # a larger token doubles the scale: the kept values are held exactly
    c, s = R.append(c, s, np.array([[[600.0, 0.0]]]), [0, 1], [1], t)
    assert s[2, 0] == 2.0 and list(R.decode(c[2, 0, 0]) * 2) == [448.0, -1.0]
    # a smaller one does not
    c2, s2 = R.append(c, s, np.array([[[1.0, 0.0]]]), [0, 1], [2], t)
    assert s2[2, 0] == 2.0 and np.array_equal(c2[2, 0, :2], c[2, 0, :2]) and R.decode(c2[2, 0, 2, 0]) == 0.5
    # a block that starts with a new token takes a scale of its own
    c3, s3 = R.append(c, s, np.array([[[1.0, 0.0]]]), [0, 1], [16], t)
    assert s3[0, 0] == 2.0 ** -8 and s3[2, 0] == 2.0 and R.decode(c3[0, 0, 0, 0]) == 256.0
    # an old scale that is no power of two is rounded up to one
    s[2, 0] = 3.0
    c4, s4 = R.append(c, s, np.array([[[1.0, 0.0]]]), [0, 1], [1], t)
    assert s4[2, 0] == 4.0 and R.decode(c4[2, 0, 0, 0]) == 160.0  # 224 * 3 / 4 = 168: a tie of 160 (1.25 * 2^7, mantissa 2) and 176, to the even code


def test_windowed_attention_against_the_whole():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((4, 2, 16, 64)), rng.standard_normal((4, 2, 16, 64))
    q = rng.standard_normal((5, 4, 64))
    t = [[3, 1, 0]]
    whole = R.attention(k, v, q, [0, 5], [30], t, 4, 0.2)
    wide = R.attention(k, v, q, [0, 5], [30], t, 4, 0.2, window=35, sinks=0)
    assert np.array_equal(whole[0], wide[0])
    ref, ref_lse = ref_numpy.paged_extend(k.astype(np.float16).view(np.uint16), v.astype(np.float16).view(np.uint16), 0, 1, 1,
                                          q.astype(np.float16).view(np.uint16), 0, [0, 5], [30], t, 4, 0.2)
    h = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    o, l, _ = R.attention(h(k), h(v), h(q), [0, 5], [30], t, 4, 0.2)
    assert np.max(np.abs(o - ref)) < 1e-12 and np.max(np.abs(l - ref_lse)) < 1e-12
    # a window of one key: that key's V; all keys as sinks: the whole
    o, l, _ = R.attention(k, v, q, [0, 5], [30], t, 4, 0.2, window=1)
    for i in range(5):
        assert np.allclose(o[i, 2], v[t[0][(30 + i) // 16], 1, (30 + i) % 16])
    o, _, _ = R.attention(k, v, q, [0, 5], [30], t, 4, 0.2, window=1, sinks=100)
    assert np.array_equal(o, whole[0])
    # one sink and one key of the window: a two-key softmax
    o, _, x = R.attention(k, v, q, [0, 5], [30], t, 4, 0.2, window=1, sinks=1)
    s0, s1 = 0.2 * q[0, 0] @ k[3, 0, 0], 0.2 * q[0, 0] @ k[1, 0, 14]
    w = 1 / (1 + np.exp(s1 - s0))
    assert np.allclose(o[0, 0], w * v[3, 0, 0] + (1 - w) * v[1, 0, 14]) and x["seen"][0, 0] == 2

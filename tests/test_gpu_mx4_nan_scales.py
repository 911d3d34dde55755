"""GPU checks of decode over microscaled codes: a NaN scale of V behind scales near the end of their range."""
import numpy as np
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests.mx4_testlib import Mx4Case, decode_ref, run_decode
from tests.pkv_testlib import BF16
from tests.scaled_testlib import check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [252, 253, 254])
@pytest.mark.parametrize("d,splits,window", [(64, 1, 0), (128, 1, 0), (128, 0, 0), (128, 2, 0), (64, 1, 290), (128, 1, 290)])
def test_a_nan_scale_behind_the_largest_ones(top, d, splits, window):
    # two tokens of the first tiles have V of +-2^(top - 128), the others +-2^118, within the factors that go
    # into the weights as they are (weights are uniform, and the sums stay below 2 2^126 + 300 2^118 < 2^128);
    # then one token's scale is NaN, for dims 32 .. 63
    n = 300
    c = Mx4Case(BF16, 1, d, 16, [n, n], seed=top + d)
    c.vs[:] = 246
    c.v = torch.from_numpy((0x11 + c.rng.integers(0, 2, c.v.shape) * 0x80 + c.rng.integers(0, 2, c.v.shape) * 0x08).astype(np.uint8))
    for b in range(2):
        for t in (20, 37):
            c.vs[int(c.tables[b, t // 16]), 0, t % 16] = top
    c.cuda()
    q = torch.zeros((2, 4, d), dtype=torch.bfloat16, device="cuda")
    good, lse = run_decode(c, q, 4, [n, n], window, 4 if window else 0, splits)
    check_attention(good, lse, decode_ref(c, q, 4, [n, n], window, 4 if window else 0), BF16, d)
    for t in (150, 227, 280, 299):
        blk = int(c.tables[1, t // 16])
        kept = c.vs[blk, 0, t % 16, 1].clone()
        c.vs[blk, 0, t % 16, 1] = 255
        out, again = run_decode(c, q, 4, [n, n], window, 4 if window else 0, splits)
        c.vs[blk, 0, t % 16, 1] = kept
        assert torch.equal(out[0], good[0]) and torch.equal(again, lse), t
        assert bool(torch.isnan(out[1, :, 32:64]).all()), t
        assert torch.equal(out[1, :, :32], good[1, :, :32]) and torch.equal(out[1, :, 64:], good[1, :, 64:]), t
    assert pkv.get_device_error() == 0

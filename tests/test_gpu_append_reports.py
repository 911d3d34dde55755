"""GPU check that the block-scaled append reports every request whose rows do not lie in the call's,
however far its indptr falls, and writes none of them."""
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests.pkv_testlib import BF16
from tests.scaled_testlib import SCALED, Case, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("fall", [1, 32, 33, 34, 64, 65, 66, 200])
def test_a_falling_indptr_is_reported(bs, fall):
    # request 0 ends `fall` rows before it begins; the others hold one row each or none
    c = Case(SCALED, BF16, 2, 64, bs, [300, 300, 300], seed=fall).cuda()
    kn, vn = c.rows(210, 2).cuda(), c.rows(210, 2).cuda()
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    for qi in ([fall, 0, 0, 0], [205, 205 - fall, 205 - fall, 205 - fall]):
        for most in (1, 210):                    # units by the hint, and by the rows (searched)
            pkv.kv_append_block_scaled(c.k, c.v, c.ks, c.vs, kn, vn, ints(qi), ints([5, 0, 0]), c.bt, most)
            assert pkv.get_device_error() == 3, (qi, most)
    for a, b in zip(before, (c.k, c.v, c.ks, c.vs)):
        assert torch.equal(a, b)

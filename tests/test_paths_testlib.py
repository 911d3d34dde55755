"""The quick float64 attention of the kernel-form tests against the row-by-row one."""
import numpy as np
import pytest

from oracle import block_scaled_ref as R
from tests import paths_testlib as P


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (9, 3), (1, 40)])
def test_attention_is_the_row_by_row_one(window, sinks):
    rng = np.random.default_rng(window)
    kv, vv = rng.standard_normal((2, 9, 2, 16, 8))
    tables = rng.permutation(9).reshape(3, 3)
    ip, prefix = [0, 5, 5, 12], [30, 7, 0]
    q = rng.standard_normal((12, 6, 8))
    want = R.attention(kv, vv, q, ip, prefix, tables, 6, 0.3, window, sinks)
    got = P.attention(kv, vv, q, ip, prefix, tables, 6, 0.3, window, sinks)
    for a, b in zip((*want[:2], *want[2].values()), (*got[:2], *got[2].values())):
        np.testing.assert_allclose(b, a, rtol=1e-12, atol=1e-13)


def test_launches_reads_both_spellings():
    got = P.launches(["void pkv::(anonymous namespace)::extend_kernel<128, 2, 1, false, (bool)0, true>(CUtensorMap_st)",
                      "void pkv::<unnamed>::extend_kernel<64, 1, 1, 0, 0, 1>(CUtensorMap_st)",
                      "pkv::(anonymous namespace)::claim_kernel(int*, pkv::ExtendParams)", "void at::fill_kernel<2>()"])
    assert got == {"extend_kernel": [[128, 2, 1, 0, 0, 1], [64, 1, 1, 0, 0, 1]], "claim_kernel": [[]]}

"""The host side of the extend over microscaled codes, without a GPU: the sizes of its workspaces and the softmax
scales that it refuses."""
import ctypes

import pytest

import paged_kv_cache_285_gb300 as pkv
from paged_kv_cache_285_gb300 import build as pkv_build
from tests.test_abi import FAKE, _desc
from tests.test_mx4_abi import mx4


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


def test_workspace_of_calls_with_few_rows(lib):
    runs = lambda **kw: lib.pkv_extend_mx4_runs_workspace_bytes(ctypes.byref(mx4(**kw)))  # noqa: E731
    both = lambda **kw: lib.pkv_extend_mx4_workspace_bytes(ctypes.byref(mx4(**kw)))  # noqa: E731
    # 152 parts of 256 rows: fp32, maximum and sum, and two records
    for d in (64, 128):
        for blocks in (1, 8, 8192, 1 << 20):
            assert runs(head_dim=d, num_blocks=blocks) == 152 * (256 * (d * 4 + 8) + 32) <= both(head_dim=d, num_blocks=blocks)
    assert both(num_blocks=8192) > 2 * runs(num_blocks=8192)
    for bad in (_desc(), _desc(cache_dtype=2), mx4(head_dim=96), mx4(num_blocks=0)):
        assert lib.pkv_extend_mx4_runs_workspace_bytes(ctypes.byref(bad)) == 0
    assert lib.pkv_extend_mx4_runs_workspace_bytes(None) == 0


@pytest.mark.parametrize("window", [0, 5])
def test_softmax_scales(lib, window):
    def extend(scale):
        return lib.pkv_paged_extend_attn_mx4(ctypes.byref(mx4()), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 4, 2,
                                             4, scale, 20, 10, 100, window, 0, None, None, 0, None)

    for scale in (0.0, -0.0, -0.125, -float("inf"), float("inf"), float("nan")):
        assert extend(scale) == 1, scale

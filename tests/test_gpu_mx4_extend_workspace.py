"""GPU checks of the extend over microscaled codes with workspaces of every size: none, one too small or misaligned,
the one of calls with few rows, and the one that pages are widened into."""
import pytest
import torch

import paged_kv_cache_285_gb300 as pkv
from tests import paths_testlib as P
from tests.mx4_testlib import Mx4Case, indptr
from tests.pkv_testlib import BF16, F16, to_f64
from tests.scaled_testlib import TDT, check_attention, ints

pytestmark = pytest.mark.gpu

TAKE = 8  # of the extend kernel's template arguments: 3 is a run per CTA
MANY = ([2100], [40])  # more than 16 pairs of row tiles: widened


@pytest.mark.parametrize("hq,hkv,d,bs,act,few_rows", [  # few_rows: shared out over all SMs
    (16, 2, 64, 32, F16, ([40, 9, 0, 33, 20], [300, 3000, 50, 1500, 0])),
    (32, 8, 128, 16, BF16, ([91, 77, 95, 43, 0, 32, 58, 31], [2052, 2107, 2280, 977, 2296, 962, 2029, 780]))])
def test_sizes(hq, hkv, d, bs, act, few_rows):
    spare = 4000 // hkv
    for rows, prefix in (few_rows, MANY):
        c = Mx4Case(act, hkv, d, bs, [p + n for p, n in zip(prefix, rows)], seed=d, spare=spare).cuda()
        q = c.rows(sum(rows), hq).cuda()
        ref = P.attention(*c.values(), to_f64(q), indptr(rows), prefix, c.tables, hq, 1 / d ** 0.5, 0, 0)
        runs, both = pkv.extend_mx4_runs_workspace_bytes(c.k), pkv.extend_mx4_workspace_bytes(c.k)
        assert both > runs + 4096
        space = torch.full((both + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        few = rows is few_rows[0]
        for at, size, taken, widened in ((0, both, few, not few), (0, runs, few, False), (0, both - 1, few, False),
                                         (0, runs - 1, False, False), (16, runs, False, False), (16, both, False, False),
                                         (256, runs + 77, few, False), (0, 0, False, False)):
            space.fill_(0x5A)
            out = torch.full((q.shape[0], hq, d), float("nan"), dtype=TDT[act], device="cuda")
            lse = torch.full((q.shape[0], hq), float("nan"), device="cuda")
            _, ran = P.profiled(lambda: pkv.paged_extend_attn_mx4(
                c.k, c.v, c.ks, c.vs, q, out, ints(indptr(rows)), ints(prefix), c.bt, 1 / d ** 0.5, max(rows), max(c.lens),
                lse_out=lse, workspace=space[at:at + size]))
            check_attention(out, lse, ref, act, d, f"{at} {size} {rows}")
            assert bool((space[:at] == 0x5A).all()) and bool((space[at + size:] == 0x5A).all()), (at, size)
            used = bool((space != 0x5A).any())
            assert used == (taken or widened), (at, size, rows)
            if ran is not None:
                assert (ran["extend_kernel"][0][TAKE] == 3) == taken and any("widen" in name for name in ran) == widened, ran
    assert pkv.get_device_error() == 0

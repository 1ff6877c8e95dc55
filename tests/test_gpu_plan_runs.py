"""Plans of one id a row whose rows come in runs of one id (adapters of requests one behind another): bit-exact to
the oracle's plan, in one block and in several."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import oracle

from _gpu import assert_plan_equal, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,begin,n,tile", [(1, 0, 1, 16), (64, 0, 1, 16), (65, 3, 2, 32), (8192, 0, 16, 128), (8191, 2, 5, 32),
                                            (20000, 0, 3, 128), (70001, 1, 1000, 16)])
@pytest.mark.parametrize("order", ["runs", "one", "none", "mixed"])
def test_runs(T, begin, n, tile, order):
    say("plan of runs", T, begin, n, tile, order)
    g = torch.Generator().manual_seed(T)
    ids = {"runs": torch.randint(-1, begin + n + 2, (T // 37 + 1,), generator=g).repeat_interleave(37)[:T],
           "one": torch.full((T,), begin + n - 1), "none": torch.full((T,), -1),
           "mixed": torch.randint(-1, begin + n + 2, (T,), generator=g)}[order].to(torch.int32).view(T, 1)
    plan, ws = moe.Plan.allocate(T, 1, begin, n, tile), moe.Workspace(T, 1, n, tile)
    for _ in range(2):
        moe.moe_plan(ids.cuda(), plan, ws)
        torch.cuda.synchronize()
        assert_plan_equal(plan, oracle.plan(ids, begin, n, tile))

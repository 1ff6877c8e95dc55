"""The plan where its split of the pairs changes: pair counts around a wave's, a column's, a block's and the scan's
registers', and expert counts around the scan's lanes. Bit for bit the oracle's plan, padding included."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import oracle

from _gpu import assert_plan_equal, say

pytestmark = pytest.mark.gpu

# pairs (K = 1), local experts, tile
SHAPES = [(n, e, 16) for n in (63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 8191, 8192, 8193, 16385)
          for e in (1, 33, 128)]
SHAPES += [(8192, 1024, 128), (8193, 1024, 128), (40_000, 1024, 64), (33_000, 513, 32), (300_001, 100, 128), (1_100_000, 31, 128)]


@pytest.mark.parametrize("pairs,E,tile", SHAPES)
def test_plan(pairs, E, tile):
    say("plan columns", pairs, E, tile)
    g = torch.Generator().manual_seed(pairs + E)
    begin = 3
    idx = torch.randint(0, E + 2 * begin, (pairs, 1), generator=g, dtype=torch.int32)   # some of other ranks
    idx[pairs // 2:pairs // 2 + 600] = begin + E - 1                                    # a run of one expert
    plan, ws = moe.Plan.allocate(pairs, 1, begin, E, tile), moe.Workspace(pairs, 1, E, tile)
    for t in (plan.src, plan.tile_expert, plan.tile_ready, plan.pos):
        t.fill_(12345)
    want = oracle.plan(idx, begin, E, tile)
    for _ in range(2):                                                                   # the second on what the first left
        moe.moe_plan(idx.cuda(), plan, ws)
        torch.cuda.synchronize()
        assert_plan_equal(plan, want)
        assert bool((plan.tile_ready == 0).all())
        assert bool((plan.src[want.P:] == -1).all()) and bool((plan.tile_expert[want.P // tile:] == -1).all())
    again = moe.Plan.allocate(pairs, 1, begin, E, tile)
    moe.moe_plan_noalloc(idx.cuda(), again)
    torch.cuda.synchronize()
    assert_plan_equal(again, want)

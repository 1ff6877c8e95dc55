"""Ids at the ends of int32: rows whose id lies outside [id_begin, id_begin + n) have no adapter, also where id - id_begin leaves 32 bits."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import test_gpu_adapter as ad

from _gpu import say

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("begin", [0, 1, HIGH - 3, HIGH - 1, HIGH])
def test_ids_at_the_ends_of_int32(begin):
    say("ids at the ends", begin)
    T, n = 24, 4
    d = ad.make(T, n, 64, 72, 16, ids=[0] * T)
    far = [LOW, LOW + 1, LOW + 2, LOW + 3, LOW + 4, -1, 0, 1, 2, HIGH, HIGH - 1, HIGH - 2]
    near = [begin + e for e in range(n) if begin + e <= HIGH]
    ids = torch.tensor((far + near + far)[:T], dtype=torch.int64)
    local = torch.where((ids >= begin) & (ids < begin + n), ids - begin, -1)
    d["ids"] = local.to(torch.int32).cuda()
    want = ad.forward(d)
    got = ad.forward(dict(d, ids=ids.to(torch.int32).cuda()), id_begin=begin)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["v"], want["v"])
    none = (local < 0).cuda()
    assert none.any() and torch.equal(got["out"][none], d["base"][none]) and (got["v"][none] == 7).all()
    plan, ws = moe.Plan.allocate(T, 1, begin, n, 16), moe.Workspace(T, 1, n, 16)
    moe.moe_plan(ids.to(torch.int32).cuda().view(T, 1), plan, ws)
    by_plan = ad.forward(d, plan)
    assert torch.equal(by_plan["out"], want["out"])

"""The norm's 8-bit copy keeps the sign of a zero, as moe_dispatch's codes do: zeros of both signs among ordinary values, in a row of
zeros and where a residual cancels, with weights of both signs. Codes, scales and pool bytes are equal bit for bit."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import block as ob

from _gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("H", [128, 1152, 4096, 16384])
@pytest.mark.parametrize("with_res", [False, True])
def test_zeros_keep_their_sign(fmt, H, with_res):
    say("norm zeros", fmt, H, with_res)
    T = 33
    g = torch.Generator().manual_seed(H)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    zero = torch.rand(T, H, generator=g)
    x[zero < 0.2] = 0.0
    x[zero < 0.1] = -0.0
    x[3], x[4] = 0.0, -0.0
    res = None
    if with_res:
        res = torch.where(torch.rand(T, H, generator=g) < 0.3, -x, torch.randn(T, H, generator=g).to(torch.bfloat16))
        res[zero < 0.1] = -0.0
    w = torch.randn(H, generator=g)
    w[::7] = -0.0
    s, _, y_ref = ob.rmsnorm(x.float().numpy(), None if res is None else res.float().numpy(), w.numpy(), 1e-6)
    assert np.signbit(y_ref[y_ref == 0]).any() and not np.signbit(y_ref[y_ref == 0]).all()
    y, q = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.uint8, device="cuda")
    q_s = moe.quantized_scales(T, H, fmt)
    moe.moe_rmsnorm(x.cuda(), w.cuda(), 1e-6, y, res=None if res is None else res.cuda(), q=q, q_s=q_s, dtype=fmt)
    torch.cuda.synchronize()
    assert np.array_equal(y.float().cpu().numpy().view(np.uint32), y_ref.view(np.uint32))
    codes, scales = ob.quantize_rows(y_ref, fmt)
    assert np.array_equal(q.cpu().numpy(), codes.view(np.uint8))
    assert np.array_equal(q_s.cpu().numpy().view(np.uint8), np.ascontiguousarray(scales).view(np.uint8))
    # the pool of the bf16 rows
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    plan, ws = moe.Plan.allocate(T, 1, 0, 1, 16), moe.Workspace(T, 1, 1, 16)
    pools = []
    for rows in (y, (q, q_s)):
        pool = torch.full((plan.rows_cap, H), 0x5A, dtype=torch.uint8, device="cuda")
        pool_s = moe.quantized_scales(plan.rows_cap, H, fmt)
        moe.moe_plan(idx, plan, ws)
        if rows is y:
            moe.moe_dispatch(y, plan, pool, pool_s, 1, ws, fmt)
        else:
            moe.moe_dispatch_quantized(q, q_s, plan, pool, pool_s, 1, ws, fmt)
        torch.cuda.synchronize()
        pools.append(pool)
    assert torch.equal(*pools)

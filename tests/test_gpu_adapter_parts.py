"""How exact v is in the products. With b = 1 and base = -bf16(v) out is what the two parts of v hold beyond the first: v's own
remainder, off by at most 2^-17 of v. (The first part leaves at most 2^-8 of the power of two below v, of which the
second, 8 bits, leaves at most 2^-17.) The gradients of the factors have all of v's 24 bits."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import test_gpu_adapter as ad

from _gpu import say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def values(T):
    """fp32 numbers of all 24 bits, both signs and many magnitudes, as sums of three bf16 numbers."""
    g = torch.Generator().manual_seed(T)
    bits = torch.randint(0, 1 << 23, (T,), generator=g, dtype=torch.int32)
    v = (bits | 0x3f800000).view(torch.float32) * torch.where(torch.rand(T, generator=g) < 0.5, -1.0, 1.0)
    v = v * torch.exp2(torch.randint(-20, 20, (T,), generator=g).float())
    parts = []
    r = v.clone()
    for _ in range(3):
        parts.append((r.view(torch.int32) & -65536).view(torch.float32).to(BF16))
        r = r - parts[-1].float()
    assert (r == 0).all()
    return v, parts


@pytest.mark.parametrize("T,tile", [(64, None), (300, 16), (2000, 32), (3000, 128)])
def test_v_in_the_products(T, tile):
    say("parts of v", T, tile)
    K = N = R = 8
    v, parts = values(T)
    d = dict(x=torch.zeros(T, K, dtype=BF16), a=torch.zeros(1, R, K, dtype=BF16), b=torch.zeros(1, N, R, dtype=BF16),
             ids=torch.zeros(T, dtype=torch.int32), scale=None, ranks=None, base=torch.zeros(T, N, dtype=BF16), dout=torch.zeros(T, N, dtype=BF16))
    d["x"][:, :3] = torch.stack(parts, 1)
    d["a"][0, 0, :3] = 1
    d["b"][0, 0, 0] = 1
    d["base"][:, 0] = -v.to(BF16)
    d = {k: t if t is None else t.cuda() for k, t in d.items()}
    plan = None if tile is None else ad.make_plan(d, tile)
    o = ad.forward(d, plan)
    assert torch.equal(o["v"][:, 0].cpu(), v)
    rest = v.double() - v.to(BF16).double()
    off = (o["out"][:, 0].cpu().double() - rest).abs() / v.double().abs()
    print("largest", float(off.max()) * 2 ** 17, "of 2^-17", flush=True)
    assert off.max() <= 2.0 ** -17 and off.max() > 2.0 ** -18        # no tighter bound holds
    assert (off > 2.0 ** -18).double().mean() < 0.25
    if plan is None:
        return
    # db[0, c] = sum of dout[t, c] v[t], one row at a time
    for t in (0, 1, T // 2, T - 1):
        d["dout"].zero_()
        d["dout"][t, 3] = 1
        g = torch.empty(1, N, R, device="cuda")
        ws = torch.empty(moe.adapter_backward_workspace_bytes(T, 1, K, N, R), dtype=torch.uint8, device="cuda")
        moe.moe_adapter_backward(d["dout"], d["x"], o["v"], d["a"], d["b"], plan, ws, None, g)
        torch.cuda.synchronize()
        assert np.float32(g[0, 3, 0].item()) == np.float32(v[t].item())

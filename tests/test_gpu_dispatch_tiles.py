"""Dispatch of quantised rows by tile (many tokens, or pairs on few experts): the bits of moe_dispatch, or, where
making the rows on the CPU would take long, of the rows gathered by the plan."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import block as ob

from _gpu import say
from test_gpu_block import poisoned_pool

pytestmark = pytest.mark.gpu


def planned(T, E, begin, E_local, K, tile, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)[1].to(torch.int32)
    idx[T // 3:T // 3 + 40, 0] = -1
    plan, ws = moe.Plan.allocate(T, K, begin, E_local, tile), moe.Workspace(T, K, E_local, tile)
    moe.moe_plan(idx, plan, ws)
    return plan, ws


# fmt, T, H, E, begin, E_local, K, tile: slices of one chunk row and less, of an instruction's lanes exactly, one more,
# several instructions; rows an instruction takes from 1 to 64; one wave's rows from 1 to 8; ranks, empty experts
CASES = [("fp8", 4096, 128, 64, 0, 64, 2, 128), ("fp8", 4100, 1152, 61, 0, 61, 3, 64), ("fp8", 4097, 4096, 32, 8, 8, 4, 32),
         ("fp8", 5000, 2048, 16, 0, 16, 8, 16), ("mxfp4", 4096, 32, 8, 0, 8, 2, 128), ("mxfp4", 4099, 160, 24, 0, 24, 2, 128),
         ("mxfp4", 4096, 2080, 12, 0, 12, 2, 64), ("mxfp4", 4096, 8192, 128, 32, 32, 4, 128), ("mxfp4", 1030, 8224, 4, 0, 4, 2, 128),
         ("mxfp4", 520, 16416, 8, 0, 8, 4, 32), ("fp8", 300, 20608, 3, 0, 3, 3, 128), ("fp8", 2049, 256, 1, 0, 1, 1, 128),
         ("mxfp4", 4096, 4128, 1000, 0, 1000, 1, 16)]


@pytest.mark.parametrize("fmt,T,H,E,begin,E_local,K,tile", CASES)
def test_rows_and_scales_go_where_the_plan_says(fmt, T, H, E, begin, E_local, K, tile):
    say("dispatch by tile", fmt, T, H, E_local, K, tile)
    plan, ws = planned(T, E, begin, E_local, K, tile, T + H)
    g = torch.Generator(device="cuda").manual_seed(H)
    q = torch.randint(0, 256, (T, H), generator=g, device="cuda", dtype=torch.uint8)
    q_s = moe.quantized_scales(T, H, fmt)
    words = (H + 127) // 128
    raw = torch.randint(0, 256, (T, 4 * words), generator=g, device="cuda", dtype=torch.uint8)
    q_s.view(torch.uint8).copy_(raw)
    pool, pool_s = poisoned_pool(plan.rows_cap, H, fmt)
    pool_s.view(torch.uint8).fill_(33)
    for epoch in (5, 6):
        moe.moe_dispatch_quantized(q, q_s, plan, pool, pool_s, epoch, ws, fmt)
        torch.cuda.synchronize()
        assert moe.moe_get_error(ws) == 0
        n = int(plan.num_tiles.item())
        if epoch == 5:
            assert bool((plan.tile_ready[:n] == 5).all()) and bool((plan.tile_ready[n:] == 0).all())
        src = plan.src.long()
        real = src >= 0
        want = torch.full_like(pool, 0x5A)
        want[real] = q[src[real] // K]
        assert torch.equal(pool, want)
        # [tile][word][row] of 4 bytes
        want = torch.full((plan.rows_cap, words, 4), 33, dtype=torch.uint8, device="cuda")
        want[real] = raw.view(T, words, 4)[src[real] // K]
        want = want.view(-1, tile, words, 4).transpose(1, 2).contiguous()
        assert torch.equal(pool_s.view(torch.uint8).flatten(), want.flatten())


def test_same_bits_as_dispatch():
    say("dispatch by tile against dispatch")
    T, H, E, K, tile = 4096, 384, 40, 2, 128
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    codes, scales = (torch.from_numpy(a).cuda() for a in ob.quantize_rows(x.float().numpy(), "fp8"))
    got = []
    for quantised in (False, True):
        plan, ws = planned(T, E, 0, E, K, tile, 9)
        pool, pool_s = poisoned_pool(plan.rows_cap, H, "fp8")
        if quantised:
            moe.moe_dispatch_quantized(codes, scales, plan, pool, pool_s, 3, ws, "fp8")
        else:
            moe.moe_dispatch(x.cuda(), plan, pool, pool_s, 3, ws, "fp8")
        torch.cuda.synchronize()
        got.append((pool, pool_s, plan.tile_ready))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_small_pool_is_reported():
    """Tiles past the pool are left out, the others whole; no write behind the pool."""
    say("dispatch by tile small pool")
    T, H, E, tile = 4096, 256, 4, 128
    plan, ws = planned(T, E, 0, E, 1, tile, 4)
    q = torch.full((T, H), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.ones(T, 2, device="cuda")
    pool, pool_s = poisoned_pool(plan.rows_cap, H, "fp8")
    rows = 10 * tile
    moe.moe_dispatch_quantized(q, s, plan, pool[:rows], pool_s[:rows], 1, ws, "fp8")
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == 1
    real = plan.src[:rows] >= 0
    assert bool((pool[:rows][real] == 0x11).all()) and bool((pool[:rows][~real] == 0x5A).all()) and bool((pool[rows:] == 0x5A).all())
    assert bool((pool_s[rows:] == 33).all())
    assert bool((plan.tile_ready[:10] == 1).all()) and bool((plan.tile_ready[10:] == 0).all())

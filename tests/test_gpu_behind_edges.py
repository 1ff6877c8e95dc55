"""Adapters and the sandwich norm where they can go wrong: the gradients' chunks full to the last row, the widest and
narrowest factors, ranks out of range, infinities in the gradients, two calls at once, rows loaded ahead in
place. Tolerances are those of the operators' own tests."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import test_gpu_adapter as ad
import test_gpu_sandwich as sw

from _gpu import say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("counts", [(256,), (257, 255), (1024, 1025, 1), (2048, 0, 3), (0, 4096, 0)], ids=str)
def test_chunks_of_the_gradients_full_and_past(counts):
    say("chunks", counts)
    ids = [e for e, c in enumerate(counts) for _ in range(c)]
    d = ad.make(len(ids), len(counts), 72, 40, 16, ids=ids)
    for tile in (16, 128):
        plan = ad.make_plan(d, tile)
        o = ad.forward(d, plan)
        ad.check_backward(d, o, ad.backward(d, o, plan))


@pytest.mark.parametrize("size", [(3, 2, 32768, 8, 8), (3, 2, 8, 32768, 8), (70, 2, 32768, 8, 256), (300, 1, 8, 32768, 64)], ids=str)
def test_widest_and_narrowest(size):
    say("widths", size)
    d = ad.make(*size, ranks=True)
    if size[0] <= 64:
        ad.check_forward(d, ad.forward(d))
    for tile in (16, 128):
        plan = ad.make_plan(d, tile)
        o = ad.forward(d, plan)
        ad.check_forward(d, o)
        ad.check_backward(d, o, ad.backward(d, o, plan))


@pytest.mark.parametrize("size", [(256, 1, 264, 136, 72), (1021, 3, 520, 264, 128), (2600, 2, 136, 1032, 136), (700, 5, 72, 72, 256)], ids=str)
def test_many_rows_of_high_ranks(size):
    """Tiles of 128 with more than 64 ranks: blocks of 64 rows, v in parts."""
    say("high ranks", size)
    for ids in ("mixed", "runs"):
        d = ad.make(*size, ids=ids, ranks=ids == "mixed")
        plan = ad.make_plan(d, 128)
        o = ad.forward(d, plan)
        ad.check_forward(d, o)
        ad.check_backward(d, o, ad.backward(d, o, plan))


def test_ranks_out_of_range():
    d = ad.make(400, 4, 136, 72, 24)
    plan = ad.make_plan(d, 32)
    taken = torch.tensor([0, 0, 24, 13], dtype=torch.int32, device="cuda")
    same = dict(d, ranks=taken)
    o = ad.forward(same, plan)
    g = ad.backward(same, o, plan)
    odd = dict(d, ranks=torch.tensor([0, -7, 2 ** 31 - 1, 13], dtype=torch.int32, device="cuda"))
    p = ad.forward(odd, plan)
    h = ad.backward(odd, p, plan)
    assert torch.equal(o["out"], p["out"]) and torch.equal(o["v"], p["v"])
    assert all(torch.equal(g[k], h[k]) for k in g)
    assert (g["da"][:2] == 0).all() and (g["db"][:2] == 0).all() and (g["da"][3, 13:] == 0).all() and (g["db"][3, :, 13:] == 0).all()
    few = {k: v[:40].contiguous() if k in ("x", "base", "ids") else v for k, v in odd.items()}
    q = ad.forward(few)
    ad.check_forward(dict(few, ranks=taken), q)


@pytest.mark.parametrize("T", [200, 600])
def test_infinite_gradients_stay_with_their_adapter(T):
    d = ad.make(T, 3, 136, 264, 16, ids=[0, 1, 2] * (T // 3) + [0] * (T % 3))
    plan = ad.make_plan(d, 128)
    o = ad.forward(d, plan)
    ref = ad.backward(d, o, plan)
    d["dout"][4, 7] = float("inf")                  # of adapter 1
    d["dout"][7, 5] = float("nan")
    g = ad.backward(d, o, plan)
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[4] = rows[7] = False
    assert torch.equal(g["dx"][rows], ref["dx"][rows]) and not torch.isfinite(g["dx"][~rows].float()).any()
    for e in (0, 2):
        assert torch.equal(g["da"][e], ref["da"][e]) and torch.equal(g["db"][e], ref["db"][e])
    assert not torch.isfinite(g["da"][1]).any()
    cols = torch.ones(264, dtype=torch.bool, device="cuda")
    cols[7] = cols[5] = False
    assert torch.equal(g["db"][1][cols], ref["db"][1][cols]) and not torch.isfinite(g["db"][1][~cols]).any()


def test_two_calls_at_once():
    """Two streams, each with its own workspaces."""
    ds = [ad.make(1500, 4, 520, 264, 24, seed=s, ids="runs") for s in (1, 2)]
    plans = [ad.make_plan(d, 32) for d in ds]
    want = [ad.forward(d, p) for d, p in zip(ds, plans)]
    streams = [torch.cuda.Stream() for _ in ds]
    outs = [torch.empty_like(o["out"]) for o in want]
    wss = [torch.empty(moe.adapter_workspace_bytes(1500, 520, 24), dtype=torch.uint8, device="cuda") for _ in ds]
    torch.cuda.synchronize()
    for _ in range(8):
        for d, p, o, ws, s in zip(ds, plans, outs, wss, streams):
            moe.moe_adapter(d["x"], d["a"], d["b"], o, ws, base=d["base"], scale=d["scale"], plan=p, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w["out"]) for o, w in zip(outs, want))


@pytest.mark.parametrize("T,H", [(257, 7168), (700, 7168), (513, 4104)])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
def test_sandwich_rows_ahead_in_place(T, H, gate):
    """16 waves a row with the next row in flight: the gradients in place of what they are made from."""
    say("rows ahead", T, H, gate)
    for gdt in (BF16, torch.float32):
        d = sw.make(T, H, 3, gate=gate, gdt=gdt)
        o = sw.forward(d, "sigmoid")
        g = sw.backward(d, o, "sigmoid")
        sw.check_backward(d, o, g, "sigmoid")
        dy, d_s = d["dy"].clone(), d["d_s"].clone()
        dg = torch.empty(H, device="cuda") if gate == "channel" else d["gate"].clone()
        ws = torch.empty(moe.sandwich_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        moe.moe_sandwich_norm_backward(dy, d_s, d["x"], o["s"], d["w"], o["r2"], dy, d_s, None, ws, post_weight=d["wp"], post_rstd=o["r1"],
                                       gate=d["gate"] if gate == "channel" else dg, gate_act="sigmoid", d_gate=dg)
        torch.cuda.synchronize()
        assert torch.equal(dy, g["dx"]) and torch.equal(d_s, g["d_res"]) and torch.equal(dg, g["d_gate"])

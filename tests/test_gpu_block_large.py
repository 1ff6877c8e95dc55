"""The block's operators where offsets pass 32 bits, two calls at once, and captured backward passes."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import block as ob

from _gpu import say

pytestmark = pytest.mark.gpu


def rows_of(t, at):
    return t[at].float().cpu().numpy()


def test_norm_past_4_gib():
    """530001 x 4096: more than 2^31 values an array. The rows looked at have no others to lean on."""
    say("norm past 4 GiB")
    T, H = 530_001, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 262_143, 262_144, 524_287, 524_288, 524_289, T - 1], device="cuda")
    x.fill_(1.0)
    x[at] = torch.randn(len(at), H, generator=g, device="cuda").to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    q, q_s = torch.empty(T, H, dtype=torch.uint8, device="cuda"), moe.quantized_scales(T, H, "mxfp4")
    moe.moe_rmsnorm(x, w, 1e-6, y, rstd=rstd, q=q, q_s=q_s, dtype="mxfp4")
    torch.cuda.synchronize()
    s, r, ref = ob.rmsnorm(rows_of(x, at), None, w.cpu().numpy(), 1e-6)
    assert np.array_equal(rows_of(y, at), ref) and np.array_equal(rstd[at].cpu().numpy(), r)
    codes, scales = ob.quantize_rows(ref, "mxfp4")
    assert np.array_equal(q[at].cpu().numpy(), codes) and np.array_equal(q_s[at].cpu().numpy(), scales)
    del q, q_s
    dy = torch.zeros_like(x)
    dy[at] = torch.randn(len(at), H, generator=g, device="cuda").to(torch.bfloat16)
    dw = torch.empty(H, device="cuda")
    ws = torch.empty(moe.rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_backward(dy, x, w, rstd, y, dw, ws)
    torch.cuda.synchronize()
    f = lambda v: v.astype(np.float64)  # noqa: E731
    dx, dweight = ob.rmsnorm_backward(f(rows_of(dy, at)), f(s), f(w.cpu().numpy()), f(r))
    # bf16's half step, and fp32 sums of 4096 terms (as in test_gpu_norm)
    assert (np.abs(rows_of(y, at) - dx) <= 2.0 ** -8 * np.abs(dx) + 2.0 ** -15).all()
    assert np.abs(dw.cpu().numpy() - dweight).max() <= 2.0 ** -18 * np.abs(dweight).max()
    others = torch.tensor([2, 262_145, 524_290, T - 2], device="cuda")
    assert bool((y[others] == 0).all())


def test_router_past_4_gib():
    say("router past 4 GiB")
    T, E, K = 8_500_001, 128, 2
    l = torch.zeros(T, E, device="cuda")
    at = torch.tensor([0, 4_194_303, 4_194_304, 8_388_607, 8_388_608, 8_388_609, T - 1], device="cuda")
    rows = torch.randn(len(at), E, generator=torch.Generator().manual_seed(2))
    l[at] = rows.cuda()
    idx, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    moe.moe_router_topk(l, idx, w)
    torch.cuda.synchronize()
    ref, _ = ob.router_topk(rows.numpy(), K)
    assert np.array_equal(idx[at].cpu().numpy(), ref)
    assert idx[T - 2].tolist() == [0, 1] and w[T - 2].tolist() == [0.5, 0.5]
    dw = torch.zeros(T, K, device="cuda")
    dw[at] = torch.randn(len(at), K, generator=torch.Generator().manual_seed(3)).cuda()
    few = torch.empty(len(at), E, device="cuda")
    moe.moe_router_topk_backward(dw[at].contiguous(), l[at].contiguous(), idx[at].contiguous(), few)
    moe.moe_router_topk_backward(dw, l, idx, l)
    torch.cuda.synchronize()
    assert torch.equal(l[at], few) and bool((l[T - 2] == 0).all())


def test_dispatch_of_quantised_rows_past_4_gib():
    """A pool of 4.6 GB: 142080 rows of 32768 codes."""
    say("dispatch past 4 GiB")
    T, H, E, K, tile = 16384, 32768, 80, 8, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randint(0, 256, (T, 1), generator=g, device="cuda", dtype=torch.uint8).expand(T, H).contiguous()
    q_s = (torch.arange(T, device="cuda").float()[:, None] + torch.arange(H // 128, device="cuda") / 1024).contiguous()
    idx = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)[1].to(torch.int32)
    plan, ws = moe.Plan.allocate(T, K, 0, E, tile), moe.Workspace(T, K, E, tile)
    assert plan.rows_cap * H > 2 ** 32
    pool = torch.empty(plan.rows_cap, H, dtype=torch.uint8, device="cuda")
    pool_s = moe.quantized_scales(plan.rows_cap, H, "fp8")
    moe.moe_plan(idx, plan, ws)
    moe.moe_dispatch_quantized(q, q_s, plan, pool, pool_s, 3, ws, "fp8")
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == 0
    n = int(plan.num_tiles.item())
    assert bool((plan.tile_ready[:n] == 3).all())
    src = plan.src[: n * tile].long()
    real = src >= 0
    assert torch.equal(pool[: n * tile][real][:, [0, 1, H // 2, H - 1]], q[src[real] // K][:, [0, 1, H // 2, H - 1]])
    got = pool_s.view(-1)[: n * tile * (H // 128)].view(n, H // 128, tile).transpose(1, 2).reshape(n * tile, -1)
    assert torch.equal(got[real], q_s[src[real] // K])


def weights(E, H, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    n = lambda *s: torch.randint(118, 121, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return r(E, 2 * I, H // 2), n(E, 2 * I, H // 32), r(E, H, I // 2), n(E, H, I // 32)


def test_decode_weights_past_4_gib():
    """The last of 64 experts of 201 MB lies past 4 GiB in both matrices: as alone."""
    say("decode past 4 GiB")
    E, H, I, K = 64, 16384, 8192, 2
    w = weights(E, H, I, 5)
    assert w[0].numel() > 2 ** 32 and w[2].numel() > 2 ** 32 // 2 + 2 ** 31 // 2
    x = torch.randn(3, H, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    tw = torch.tensor([[0.5, 0.5], [1.0, 2.0], [0.25, 4.0]], device="cuda")
    idx = torch.tensor([[63, 0], [63, 62], [1, 63]], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.expert_ffn_decode_workspace_bytes(3, K, I), dtype=torch.uint8, device="cuda")
    out, ref = torch.empty(3, H, dtype=torch.bfloat16, device="cuda"), torch.empty(3, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_decode(x, None, idx, tw, *w, ws, out)
    few = [t[[0, 1, 62, 63]].contiguous() for t in w]
    small = torch.tensor([[3, 0], [3, 2], [1, 3]], dtype=torch.int32, device="cuda")
    moe.moe_expert_ffn_decode(x, None, small, tw, *few, ws, ref)
    torch.cuda.synchronize()
    assert bool((ref != 0).any()) and torch.equal(out, ref)


def test_two_calls_at_once():
    """Two streams, a workspace each: what one after the other gives."""
    say("two calls at once")
    E, H, I, K, T = 16, 2048, 512, 4, 24
    w = weights(E, H, I, 7)
    g = torch.Generator(device="cuda").manual_seed(8)
    sets = []
    for _ in range(2):
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        idx = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)[1].to(torch.int32)
        sets.append(dict(x=x, idx=idx, tw=torch.rand(T, K, generator=g, device="cuda"), out=torch.empty_like(x), dx=torch.empty_like(x),
                         dw=torch.empty(H, device="cuda"), rstd=torch.empty(T, device="cuda"), y=torch.empty_like(x),
                         dws=torch.empty(moe.expert_ffn_decode_workspace_bytes(T, K, I), dtype=torch.uint8, device="cuda"),
                         nws=torch.empty(moe.rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")))
    weight = torch.ones(H, device="cuda")

    def step(s, stream):
        moe.moe_rmsnorm(s["x"], weight, 1e-6, s["y"], rstd=s["rstd"], stream=stream)
        moe.moe_expert_ffn_decode(s["y"], None, s["idx"], s["tw"], *w, s["dws"], s["out"], stream=stream)
        moe.moe_rmsnorm_backward(s["out"], s["x"], weight, s["rstd"], s["dx"], s["dw"], s["nws"], stream=stream)

    ref = []
    for s in sets:
        step(s, None)
        torch.cuda.synchronize()
        ref.append([s[n].clone() for n in ("out", "dx", "dw")])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s in sets:
            for n in ("out", "dx", "dw"):
                s[n].zero_()
        torch.cuda.synchronize()
        for s, stream in zip(sets, streams):
            step(s, stream)
        torch.cuda.synchronize()
        for s, r in zip(sets, ref):
            assert all(torch.equal(s[n], v) for n, v in zip(("out", "dx", "dw"), r))


def test_captured_backward_replays():
    say("captured backward")
    T, H, E, K = 700, 1024, 48, 4
    cfg = moe.RouterConfig(score="sigmoid", groups=4, topk_groups=2, group_top=2)
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
    x, dy, w = e(T, H, dtype=torch.bfloat16), e(T, H, dtype=torch.bfloat16), torch.ones(H, device="cuda")
    logits, dtw = e(T, E), e(T, K)
    ws = e(moe.rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8)

    def step():
        o = dict(y=e(T, H, dtype=torch.bfloat16), rstd=e(T), dx=e(T, H, dtype=torch.bfloat16), dw=e(H),
                 idx=e(T, K, dtype=torch.int32), tw=e(T, K), dl=e(T, E))
        moe.moe_rmsnorm(x, w, 1e-6, o["y"], rstd=o["rstd"])
        moe.moe_rmsnorm_backward(dy, x, w, o["rstd"], o["dx"], o["dw"], ws)
        moe.moe_router_topk(logits, o["idx"], o["tw"], cfg)
        moe.moe_router_topk_backward(dtw, logits, o["idx"], o["dl"], cfg)
        return o

    for t in (x, dy, logits, dtw):
        t.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t in (x, dy, logits, dtw):
            t.normal_(generator=torch.Generator(device="cuda").manual_seed(i))
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        torch.cuda.synchronize()
        for n, v in ref.items():
            assert torch.equal(got[n], v), (i, n)


def test_layer_refuses_rows_of_another_kind():
    say("layer refusals")
    q, s = torch.zeros(8, 512, dtype=torch.uint8, device="cuda"), torch.ones(8, 4, device="cuda")
    idx, tw = torch.zeros(8, 2, dtype=torch.int32, device="cuda"), torch.ones(8, 2, device="cuda")
    layer = moe.StreamMoE(8, 512, 256, 2, 4, dtype="bf16")
    w = torch.zeros(4, 512, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 512, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError):
        layer.forward((q, s), idx, tw, *w)
    layer = moe.StreamMoE(8, 512, 256, 2, 4, dtype="mxfp4")
    with pytest.raises(ValueError):              # fp8 scales in front of an mxfp4 layer
        layer.forward((q, s), idx, tw, *w)
    with pytest.raises(ValueError):              # another number of rows
        layer.forward((q[:5], s[:5]), idx, tw, *w)
    big = moe.StreamMoE(80, 512, 256, 2, 4, dtype="mxfp4")
    wp = big.prepare_weights(*(torch.zeros(*z, dtype=torch.uint8, device="cuda") for z in
                               ((4, 512, 256), (4, 512, 128), (4, 512, 16), (4, 512, 8))))
    x = torch.zeros(65, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError):            # more tokens than decode takes
        big.decode(x, torch.zeros(65, 2, dtype=torch.int32, device="cuda"), torch.ones(65, 2, device="cuda"), *wp)
    out = big.decode(x[:64], torch.zeros(64, 2, dtype=torch.int32, device="cuda"), torch.ones(64, 2, device="cuda"), *wp)
    torch.cuda.synchronize()
    assert bool((out == 0).all())

"""The operators around the layer, run together as a transformer's MoE block runs them: the norm's
8-bit rows through dispatch and the experts (bit for bit what the bf16 rows give), the serving
chain of a few tokens eager, captured and on another stream, and the training chain's gradients
against a float64 model of the block."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import combine_moe_dispatch_02_amd as moe
import oracle
from oracle import block as ob
from synth import MoEConfig, make_inputs

from _gpu import make_layer, say

pytestmark = pytest.mark.gpu


def poisoned_pool(rows, H, fmt):
    pool = torch.full((rows, H), 0x5A, dtype=torch.uint8, device="cuda")
    return pool, moe.quantized_scales(rows, H, fmt).fill_(33)


DISPATCH = [("fp8", 64, 128, 8, 0, 8, 2, 16), ("fp8", 700, 1152, 16, 0, 16, 4, 128), ("fp8", 33, 4096, 24, 8, 8, 8, 32),
            ("fp8", 1, 7168, 8, 0, 8, 8, 64), ("mxfp4", 64, 32, 8, 0, 8, 2, 16), ("mxfp4", 700, 160, 16, 0, 16, 4, 128),
            ("mxfp4", 257, 2080, 24, 8, 8, 16, 64), ("mxfp4", 1, 4096, 8, 2, 2, 3, 128), ("mxfp4", 5, 16416, 8, 0, 8, 1, 32),
            ("fp8", 9001, 256, 61, 0, 61, 5, 128)]


@pytest.mark.parametrize("fmt,T,H,E,begin,E_local,K,tile", DISPATCH)
def test_dispatch_of_quantised_rows_is_dispatch(fmt, T, H, E, begin, E_local, K, tile):
    say("dispatch quantised", fmt, T, H, K)
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    idx = torch.rand(T, E, generator=g).topk(min(K, E), dim=1)[1].to(torch.int32)
    idx = torch.cat([idx, torch.full((T, K - idx.shape[1]), -1, dtype=torch.int32)], 1).contiguous().cuda()
    codes, scales = ob.quantize_rows(x.float().numpy(), fmt)
    got = []
    for quantised in (False, True):
        plan = moe.Plan.allocate(T, K, begin, E_local, tile)
        ws = moe.Workspace(T, K, E_local, tile)
        pool, pool_s = poisoned_pool(plan.rows_cap, H, fmt)
        moe.moe_plan(idx, plan, ws)
        if quantised:
            moe.moe_dispatch_quantized(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), plan, pool, pool_s, 5, ws,
                                       fmt)
        else:
            moe.moe_dispatch(x.cuda(), plan, pool, pool_s, 5, ws, fmt)
        torch.cuda.synchronize()
        assert moe.moe_get_error(ws) == 0
        n = int(plan.num_tiles.item())
        assert bool((plan.tile_ready[:n] == 5).all())
        got.append((pool, pool_s, plan.tile_ready.clone()))
    for name, a, b in zip(("pool", "scales", "flags"), *got):
        if name == "scales" and fmt == "mxfp4" and H % 128:
            # bytes past a row's last block: dispatch leaves them, a quantised row brings zeros; neither is read
            blocks = H // 32 % 4
            a = a.reshape(-1, (H + 127) // 128, tile, 4)
            b = b.reshape(a.shape)
            assert torch.equal(a[:, :-1], b[:, :-1])
            a, b = a[:, -1, :, :blocks], b[:, -1, :, :blocks]
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), name


def test_dispatch_of_quantised_rows_reports_a_small_pool():
    say("dispatch quantised small pool")
    T, H, E = 64, 128, 4
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    plan, ws = moe.Plan.allocate(T, 1, 0, E, 16), moe.Workspace(T, 1, E, 16)
    moe.moe_plan(idx, plan, ws)
    pool, pool_s = poisoned_pool(64, H, "fp8")
    q = torch.full((T, H), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.ones(T, 1, device="cuda")
    moe.moe_dispatch_quantized(q, s, plan, pool[:32], pool_s[:32], 1, ws, "fp8")
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == 1 and bool((pool[:32] == 0x11).all()) and bool((pool[32:] == 0x5A).all())
    with pytest.raises(ValueError):
        moe.moe_dispatch_quantized(q, s, plan, pool, pool_s[:32], 1, ws, "fp8")
    with pytest.raises(ValueError):
        moe.moe_dispatch_quantized(q, s[:5], plan, pool, pool_s, 1, ws, "fp8")
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch_quantized(q, s, plan, pool, pool_s, 1, ws, "bf16")


PROMPT = [MoEConfig("blk_fp8", 300, 512, 256, 6, 0, 6, 2, 64, "fp8"), MoEConfig("blk_fp8_big", 600, 1024, 512, 12, 2, 8, 4, 128, "fp8"),
          MoEConfig("blk_mx", 600, 1024, 512, 12, 2, 8, 4, 128, "mxfp4")]


def block_inputs(cfg, seed=3):
    inp = make_inputs(cfg, seed)
    g = torch.Generator().manual_seed(seed)
    d = dict(x=inp.x.cuda(), res=torch.randn(cfg.T, cfg.H, generator=g).to(torch.bfloat16).cuda(),
             norm=(1 + 0.1 * torch.randn(cfg.H, generator=g)).cuda(),
             wr=(torch.randn(cfg.num_experts, cfg.H, generator=g) / cfg.H ** 0.5).cuda())
    return inp, d


def gate(d, y):
    """The router's logits: a plain product (float64, so that they do not hang on a library's order)."""
    return (y.double() @ d["wr"].double().t()).float()


@pytest.mark.parametrize("streams", [False, True])
@pytest.mark.parametrize("cfg", PROMPT, ids=lambda c: c.name)
def test_prompt_through_quantised_rows(cfg, streams):
    say("block prompt", cfg.name, streams)
    inp, d = block_inputs(cfg)
    layer = make_layer(cfg)
    w = layer.prepare_weights(*(t.view(torch.uint8).cuda() if t.dtype != torch.float32 else t.cuda()
                                for t in (inp.w1, inp.w2, inp.w1_scale, inp.w2_scale)))
    y, s = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    q, q_s = torch.empty(cfg.T, cfg.H, dtype=torch.uint8, device="cuda"), moe.quantized_scales(cfg.T, cfg.H, cfg.dtype)
    moe.moe_rmsnorm(d["x"], d["norm"], 1e-6, y, res=d["res"], res_out=s, q=q, q_s=q_s, dtype=cfg.dtype)
    idx = torch.empty(cfg.T, cfg.K, dtype=torch.int32, device="cuda")
    tw = torch.empty(cfg.T, cfg.K, device="cuda")
    moe.moe_router_topk(gate(d, y), idx, tw)
    st = moe.make_streams() if streams else None
    a = layer.forward(y, idx, tw, *w, streams=st).clone()
    b = layer.forward((q, q_s), idx, tw, *w, streams=st)
    torch.cuda.synchronize()
    layer.check_errors()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and bool((a != 0).any())


class Serving:
    """One block's buffers and weights for up to T tokens."""

    def __init__(self, cfg):
        self.cfg = cfg
        self.inp, self.d = block_inputs(cfg)
        self.layer = make_layer(cfg)
        self.w = self.layer.prepare_weights(*(t.view(torch.uint8).cuda() for t in
                                              (self.inp.w1, self.inp.w2, self.inp.w1_scale, self.inp.w2_scale)))
        T, H = cfg.T, cfg.H
        self.y, self.s = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        self.q, self.q_s = torch.empty(T, H, dtype=torch.uint8, device="cuda"), moe.quantized_scales(T, H, "mxfp4")
        self.idx = torch.empty(T, cfg.K, dtype=torch.int32, device="cuda")
        self.tw = torch.empty(T, cfg.K, device="cuda")
        self.wr = self.d["wr"].t().contiguous()

    def step(self, x, res):
        moe.moe_rmsnorm(x, self.d["norm"], 1e-6, self.y, res=res, res_out=self.s, q=self.q, q_s=self.q_s, dtype="mxfp4")
        logits = (self.y.float().unsqueeze(2) * self.wr).sum(1)      # elementwise: safe to capture
        moe.moe_router_topk(logits, self.idx, self.tw, moe.RouterConfig(score="sigmoid", groups=4, topk_groups=2, group_top=2))
        return self.layer.decode((self.q, self.q_s), self.idx, self.tw, *self.w)


@pytest.mark.parametrize("T", [1, 5, 24])
def test_serving_chain_eager_captured_and_on_another_stream(T):
    say("block serving", T)
    cfg = MoEConfig("serve", T, 512, 256, 16, 4, 8, 4, 128, "mxfp4")
    eager, graphed = Serving(cfg), Serving(cfg)
    x, res = eager.d["x"].clone(), eager.d["res"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(x, res)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = graphed.step(x, res)
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        x.copy_(torch.randn(T, 512, generator=gen, device="cuda"))
        res.copy_(torch.randn(T, 512, generator=gen, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        ref = eager.step(x.clone(), res.clone()).clone()
        torch.cuda.synchronize()
        for a, b in ((out, ref), (graphed.s, eager.s), (graphed.idx, eager.idx), (graphed.tw, eager.tw)):
            assert torch.equal(a, b), i
        # on another stream, the inputs made there
        with torch.cuda.stream(side):
            other = eager.step(x.clone(), res.clone()).clone()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(other, ref)
    # against the oracle, on the last inputs and the chosen experts
    y = ob.rmsnorm(x.float().cpu().numpy(), res.float().cpu().numpy(), eager.d["norm"].cpu().numpy(), 1e-6)[2]
    inp = eager.inp
    want = ob.expert_ffn_decode(y, None, eager.idx.cpu().numpy(), eager.tw.cpu().numpy(),
                                *(t.view(torch.uint8).numpy() for t in (inp.w1, inp.w1_scale, inp.w2, inp.w2_scale)),
                                expert_begin=4)
    assert oracle.max_norm_rel_err(oracle.bf16_to_f64(out.cpu()), want) <= 3e-2


def test_stream_and_device_checks():
    say("block streams")
    x = torch.randn(3, 256, device="cuda").to(torch.bfloat16)
    w, y = torch.ones(256, device="cuda"), torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        y.fill_(0)
        torch.cuda.synchronize()
        moe.moe_rmsnorm(x, w, 1e-6, y, stream=stream)
        side.synchronize()
        assert bool((y != 0).any())


def test_training_chain_gradients():
    """Forward and backward of the whole block. The float64 model takes the kernels' choice of
    experts; everything else it computes from the inputs. A chain of about ten bf16 roundings
    (stream, y, pool, G, h, y_pool, out, dy, dG, dx; 2^-9 rms each) stays within 3e-2 of the
    largest value."""
    say("block training")
    cfg = MoEConfig("train", 192, 512, 512, 6, 0, 6, 2, 64)
    inp, d = block_inputs(cfg, 9)
    T, H, K, E = cfg.T, cfg.H, cfg.K, cfg.num_experts
    rcfg = moe.RouterConfig(score="sigmoid", scale=1.5)
    layer = make_layer(cfg, train=True)
    w1, w2 = inp.w1.cuda(), inp.w2.cuda()
    w = layer.prepare_weights(w1, w2)
    wt = layer.prepare_backward_weights(w1, w2)
    bf = lambda: torch.empty(T, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    s, y, dx = bf(), bf(), bf()
    rstd = torch.empty(T, device="cuda")
    moe.moe_rmsnorm(d["x"], d["norm"], 1e-6, y, res=d["res"], res_out=s, rstd=rstd)
    logits = gate(d, y)
    idx, tw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    moe.moe_router_topk(logits, idx, tw, rcfg)
    out = layer.forward(y, idx, tw, w[0], w[1]).clone()
    d_out = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    dyl, dtw, dw1, dw2 = layer.backward(d_out, tw, *wt)
    d_logits = torch.empty_like(logits)
    moe.moe_router_topk_backward(dtw, logits, idx, d_logits, rcfg)
    dy = (dyl.float() + d_logits @ d["wr"]).to(torch.bfloat16)
    d_norm = torch.empty(H, device="cuda")
    ws = torch.empty(moe.rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_backward(dy, s, d["norm"], rstd, dx, d_norm, ws, d_res=d_out)   # block output: s + out
    torch.cuda.synchronize()
    layer.check_errors()

    f = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
    x6, n6, r6, W1, W2 = f(d["x"].double() + d["res"].double()), f(d["norm"]), f(d["wr"]), f(inp.w1), f(inp.w2)
    y6 = x6 / torch.sqrt(x6.square().mean(1, keepdim=True) + 1e-6) * n6
    sc = torch.sigmoid(y6 @ r6.t()).gather(1, idx.cpu().long())
    t6 = sc / sc.sum(1, keepdim=True) * 1.5
    o6 = torch.zeros(T, H, dtype=torch.float64)
    for k in range(K):
        for e in range(E):
            m = (idx[:, k] == e).cpu()
            if m.any():
                G = y6[m] @ W1[e].t()
                o6 = o6.index_add(0, m.nonzero().squeeze(1), t6[m, k:k + 1] * ((F.silu(G[:, :512]) * G[:, 512:]) @ W2[e].t()))
    ((x6 + o6) * d_out.cpu().double()).sum().backward()
    for name, got, ref in (("out", out, o6), ("dx", dx, x6.grad), ("dnorm", d_norm, n6.grad), ("dw1", dw1, W1.grad),
                           ("dw2", dw2, W2.grad), ("dwr", d_logits.double().t() @ y.double(), r6.grad)):
        err = oracle.max_norm_rel_err(got.detach().cpu().double().numpy(), ref.detach().numpy())
        assert err <= 3e-2, (name, err)

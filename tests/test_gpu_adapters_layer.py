"""The layer with low-rank adapters and the sandwich norm behind it, run together as a fine-tuned
block runs them: with adapters the layer gives, bit for bit, what moe_adapter adds to its output; a
serving chain eager, captured and on another stream; a training chain's gradients against a
float64 model of the block."""
import pytest
import torch
import torch.nn.functional as F

import combine_moe_dispatch_02_amd as moe
import oracle
from oracle import behind as oh
from oracle import block as ob
from synth import MoEConfig, make_inputs

from _gpu import make_layer, say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def adapters_of(T, n, H, R, seed, train=False, ids=None):
    g = torch.Generator().manual_seed(seed)
    a, b = (torch.randn(n, R, H, generator=g) / H ** 0.5).to(BF16).cuda(), (torch.randn(n, H, R, generator=g) / R ** 0.5).to(BF16).cuda()
    scale = (0.5 + torch.rand(n, generator=g)).cuda()
    if ids is None:
        ids = torch.randint(-1, n, (T,), generator=g)
    rows = moe.AdapterRows(T, n, train=train).set(ids.to(torch.int32).cuda())
    return moe.Adapters(a, b, rows, scale=scale, train=train)


@pytest.mark.parametrize("mode", ["one stream", "two streams", "combine on completion"])
@pytest.mark.parametrize("T", [48, 300])
def test_layer_adds_its_rows_adapters(mode, T):
    say("layer with adapters", mode, T)
    cfg = MoEConfig("ad", T, 512, 512, 6, 0, 6, 2, 64)
    inp = make_inputs(cfg, 4)
    layer = make_layer(cfg, combine_on_completion=mode == "combine on completion")
    w = layer.prepare_weights(inp.w1.cuda(), inp.w2.cuda())
    x, idx, tw = inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_weights.cuda()
    st = moe.make_streams() if mode == "two streams" else None
    ad = adapters_of(T, 5, 512, 24, T)
    plain = layer.forward(x, idx, tw, w[0], w[1], streams=st).clone()
    want = ad.add(x, plain, torch.empty_like(plain))
    got = layer.forward(x, idx, tw, w[0], w[1], streams=st, adapters=ad)
    torch.cuda.synchronize()
    layer.check_errors()
    assert torch.equal(got, want) and not torch.equal(got, plain)
    ids = ad.rows.ids.cpu().numpy()
    ref, _ = oh.adapter(x.double().cpu().numpy(), ids, ad.a.double().cpu().numpy(), ad.b.double().cpu().numpy(),
                        ad.scale.double().cpu().numpy(), None, plain.double().cpu().numpy())
    assert oracle.max_norm_rel_err(oracle.bf16_to_f64(got.cpu()), ref) <= 2.0 ** -8


@pytest.mark.parametrize("streams", [False, True])
def test_layer_gradients_have_the_adapters_share(streams):
    say("layer gradients with adapters", streams)
    T = 192
    cfg = MoEConfig("adtrain", T, 512, 512, 6, 0, 6, 2, 64)
    inp = make_inputs(cfg, 5)
    layer = make_layer(cfg, train=True)
    w1, w2 = inp.w1.cuda(), inp.w2.cuda()
    w, wt = layer.prepare_weights(w1, w2), layer.prepare_backward_weights(w1, w2)
    x, idx, tw = inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_weights.cuda()
    dout = torch.randn(T, 512, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    st = moe.make_streams() if streams else None
    ad, by_hand = adapters_of(T, 3, 512, 16, 7, train=True), adapters_of(T, 3, 512, 16, 7, train=True)
    layer.forward(x, idx, tw, w[0], w[1], streams=st)
    plain = [t.clone() for t in layer.backward(dout, tw, *wt, streams=st)]
    by_hand.add(x, torch.zeros_like(dout))
    dx = torch.empty_like(x)
    by_hand.backward(dout, plain[0], dx)
    layer.forward(x, idx, tw, w[0], w[1], streams=st, adapters=ad)
    got = layer.backward(dout, tw, *wt, streams=st, adapters=ad)
    torch.cuda.synchronize()
    layer.check_errors()
    assert torch.equal(got[0], dx) and torch.equal(ad.da, by_hand.da) and torch.equal(ad.db, by_hand.db)
    assert all(torch.equal(p, q) for p, q in zip(plain[1:], got[1:]))


def test_refusals():
    say("adapters refused")
    cfg = MoEConfig("serve", 4, 512, 256, 16, 0, 16, 4, 128, "mxfp4")
    inp = make_inputs(cfg, 1)
    layer = make_layer(cfg)
    w = layer.prepare_weights(*(t.view(torch.uint8).cuda() for t in (inp.w1, inp.w2, inp.w1_scale, inp.w2_scale)))
    idx, tw = inp.topk_idx.cuda(), inp.topk_weights.cuda()
    q, q_s = torch.zeros(4, 512, dtype=torch.uint8, device="cuda"), moe.quantized_scales(4, 512, "mxfp4").zero_()
    ad = adapters_of(4, 2, 512, 8, 1)
    for call in (layer.forward, layer.decode):
        with pytest.raises(ValueError, match="bf16 rows"):
            call((q, q_s), idx, tw, *w, adapters=ad)
        with pytest.raises(ValueError, match="do not match"):
            call((q, q_s), idx, tw, *w, adapters=ad, adapter_x=torch.zeros(3, 512, dtype=BF16, device="cuda"))
        with pytest.raises(ValueError, match="do not match"):
            call((q, q_s), idx, tw, *w, adapters=adapters_of(4, 2, 256, 8, 1), adapter_x=torch.zeros(4, 512, dtype=BF16, device="cuda"))
    with pytest.raises(RuntimeError, match="set"):
        moe.Adapters(ad.a, ad.b, moe.AdapterRows(4, 2)).add(torch.zeros(4, 512, dtype=BF16, device="cuda"), q.to(BF16))
    with pytest.raises(ValueError, match="ids"):
        moe.AdapterRows(4, 2).set(torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="adapters"):
        moe.Adapters(ad.a, ad.b, moe.AdapterRows(4, 3))
    with pytest.raises(ValueError, match="train"):
        moe.Adapters(ad.a, ad.b, moe.AdapterRows(4, 2), train=True)
    with pytest.raises(RuntimeError, match="add"):
        ad.backward(q.to(BF16), None)
    with pytest.raises(ValueError, match="do not match|shape"):
        ad.add(torch.zeros(5, 512, dtype=BF16, device="cuda"), torch.zeros(5, 512, dtype=BF16, device="cuda"))


def test_no_rows_and_rows_left_alone():
    """A batch without rows: gradients of zero. A row without an adapter: its v stays as it was."""
    say("adapters of no rows")
    a, b = torch.zeros(2, 8, 64, dtype=BF16, device="cuda"), torch.zeros(2, 64, 8, dtype=BF16, device="cuda")
    ad = moe.Adapters(a, b, moe.AdapterRows(0, 2, train=True).set(torch.empty(0, dtype=torch.int32, device="cuda")), train=True)
    none = torch.empty(0, 64, dtype=BF16, device="cuda")
    ad.da.fill_(7), ad.db.fill_(7)
    ad.add(none, none)
    ad.backward(none, none)
    torch.cuda.synchronize()
    assert (ad.da == 0).all() and (ad.db == 0).all()
    for T in (40, 400):
        ids = torch.arange(T) % 3 - 1
        ad = adapters_of(T, 2, 256, 16, 3, train=True, ids=ids)
        ad.v.fill_(7.0)
        x = torch.randn(T, 256, device="cuda").to(BF16)
        ad.add(x, torch.zeros_like(x))
        torch.cuda.synchronize()
        assert (ad.v[ids.cuda() < 0] == 7).all() and (ad.v[ids.cuda() >= 0] != 7).any(1).all()


class Serving:
    """One block of up to T tokens: norm, router, MXFP4 experts with adapters, and the norm of what they give in front of
    the next block, which takes MXFP8 rows."""

    def __init__(self, cfg, n):
        T, H = cfg.T, cfg.H
        self.inp, g = make_inputs(cfg, 3), torch.Generator().manual_seed(8)
        self.norm, self.post = (1 + 0.1 * torch.randn(H, generator=g)).cuda(), (0.8 + 0.1 * torch.randn(H, generator=g)).cuda()
        self.wr = (torch.randn(H, cfg.num_experts, generator=g) / H ** 0.5).cuda()
        self.gate = torch.randn(T, 1, generator=g).cuda()
        self.layer = make_layer(cfg)
        self.w = self.layer.prepare_weights(*(t.view(torch.uint8).cuda() for t in
                                              (self.inp.w1, self.inp.w2, self.inp.w1_scale, self.inp.w2_scale)))
        self.ad = adapters_of(T, n, H, 16, 11, ids=torch.arange(T) % (n + 1) - 1)
        bf = lambda: torch.empty(T, H, dtype=BF16, device="cuda")  # noqa: E731
        self.y, self.s, self.y2, self.s2 = bf(), bf(), bf(), bf()
        self.q, self.q_s = torch.empty(T, H, dtype=torch.uint8, device="cuda"), moe.quantized_scales(T, H, "mxfp4")
        self.idx, self.tw = torch.empty(T, cfg.K, dtype=torch.int32, device="cuda"), torch.empty(T, cfg.K, device="cuda")

    def step(self, x, res):
        moe.moe_rmsnorm(x, self.norm, 1e-6, self.y, res=res, res_out=self.s, q=self.q, q_s=self.q_s, dtype="mxfp4")
        logits = (self.y.float().unsqueeze(2) * self.wr).sum(1)      # elementwise: safe to capture
        moe.moe_router_topk(logits, self.idx, self.tw)
        out = self.layer.decode((self.q, self.q_s), self.idx, self.tw, *self.w, adapters=self.ad, adapter_x=self.y)
        moe.moe_sandwich_norm(out, self.s, self.norm, 1e-6, self.s2, self.y2, post_weight=self.post, gate=self.gate, gate_act="sigmoid",
                              q=self.q, q_s=self.q_s, dtype="mxfp4")
        return out


@pytest.mark.parametrize("T", [1, 5, 24])
def test_serving_chain_eager_captured_and_on_another_stream(T):
    say("serving with adapters", T)
    cfg = MoEConfig("serve", T, 512, 256, 16, 4, 8, 4, 128, "mxfp4")
    eager, graphed = Serving(cfg, 3), Serving(cfg, 3)
    x, res = torch.empty(T, 512, dtype=BF16, device="cuda"), torch.empty(T, 512, dtype=BF16, device="cuda")
    x.normal_(), res.normal_()
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
        for a, b in ((out, ref), (graphed.s2, eager.s2), (graphed.y2, eager.y2), (graphed.q, eager.q), (graphed.q_s, eager.q_s)):
            assert torch.equal(a, b), i
        with torch.cuda.stream(side):
            other = eager.step(x.clone(), res.clone()).clone()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(other, ref)
    # what the adapters and the norm did with what they had, in float64 (a bf16 rounding each)
    inp, n64 = eager.inp, lambda t: t.double().cpu().numpy()  # noqa: E731
    experts = ob.expert_ffn_decode(n64(eager.y).astype("float32"), None, eager.idx.cpu().numpy(), eager.tw.cpu().numpy(),
                                   *(t.view(torch.uint8).numpy() for t in (inp.w1, inp.w1_scale, inp.w2, inp.w2_scale)), expert_begin=4)
    want, _ = oh.adapter(n64(eager.y), eager.ad.rows.ids.cpu().numpy(), n64(eager.ad.a), n64(eager.ad.b), n64(eager.ad.scale), None, experts)
    assert oracle.max_norm_rel_err(oracle.bf16_to_f64(out.cpu()), want) <= 3e-2
    s, _, _ = oh.sandwich(n64(out), n64(eager.s), n64(eager.post), n64(eager.gate), "sigmoid", 1.0, 1.0, 1e-6)
    assert oracle.max_norm_rel_err(oracle.bf16_to_f64(eager.s2.cpu()), s) <= 2.0 ** -8
    _, y2 = oh.sandwich_norm(n64(eager.s2).astype("float32"), n64(eager.norm).astype("float32"), 1e-6)
    codes, scales = ob.quantize_rows(y2, "mxfp4")
    assert (eager.q.cpu().numpy() == codes).all() and (eager.q_s.cpu().numpy() == scales).all()


def test_training_chain_gradients():
    """Forward and backward of a block with adapters beside the experts and the sandwich norm behind them, against a
    float64 model that takes the kernels' choice of experts. A chain of about a dozen bf16 roundings (2^-9 rms
    each) stays within 3e-2 of the largest value."""
    say("training with adapters")
    cfg = MoEConfig("train", 192, 512, 512, 6, 0, 6, 2, 64)
    T, H, K, E, n, R = cfg.T, cfg.H, cfg.K, cfg.num_experts, 3, 16
    inp, gen = make_inputs(cfg, 9), torch.Generator().manual_seed(6)
    layer = make_layer(cfg, train=True)
    w1, w2 = inp.w1.cuda(), inp.w2.cuda()
    w, wt = layer.prepare_weights(w1, w2), layer.prepare_backward_weights(w1, w2)
    x, idx, tw = inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_weights.cuda()
    res = torch.randn(T, H, generator=gen).to(BF16).cuda()
    post, norm = (0.8 + 0.1 * torch.randn(H, generator=gen)).cuda(), (1 + 0.1 * torch.randn(H, generator=gen)).cuda()
    gate = (0.5 * torch.randn(H, generator=gen)).cuda()
    ad = adapters_of(T, n, H, R, 13, train=True)
    bf, f32 = lambda: torch.empty(T, H, dtype=BF16, device="cuda"), lambda k: torch.empty(k, device="cuda")  # noqa: E731
    s, y, r1, r2 = bf(), bf(), f32(T), f32(T)
    kw = dict(post_weight=post, gate=gate, gate_act="tanh", res_scale=0.9, branch_scale=1.2)
    out = layer.forward(x, idx, tw, w[0], w[1], adapters=ad)
    moe.moe_sandwich_norm(out, res, norm, 1e-6, s, y, **kw, post_rstd=r1, rstd=r2)
    dy, d_s = (torch.randn(T, H, generator=gen).to(BF16).cuda() for _ in range(2))
    d_out, d_res, d_norm, d_post, d_gate = bf(), bf(), f32(H), f32(H), f32(H)
    ws = torch.empty(moe.sandwich_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_sandwich_norm_backward(dy, d_s, out, s, norm, r2, d_out, d_res, d_norm, ws, post_rstd=r1, **kw, d_post_weight=d_post, d_gate=d_gate)
    dx, _, dw1, dw2 = layer.backward(d_out, tw, *wt, adapters=ad)
    torch.cuda.synchronize()
    layer.check_errors()

    f = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
    x6, s6, p6, n6, g6, W1, W2, A6, B6 = (f(t) for t in (x, res, post, norm, gate, inp.w1, inp.w2, ad.a, ad.b))
    t6, i6, ids = tw.cpu().double(), idx.cpu(), ad.rows.ids.cpu()
    o6 = torch.zeros(T, H, dtype=torch.float64)
    for k in range(K):
        for e in range(E):
            m = i6[:, k] == e
            if m.any():
                G = x6[m] @ W1[e].t()
                o6 = o6.index_add(0, m.nonzero().squeeze(1), t6[m, k:k + 1] * ((F.silu(G[:, :512]) * G[:, 512:]) @ W2[e].t()))
    for e in range(n):
        m = ids == e
        o6 = o6.index_add(0, m.nonzero().squeeze(1), float(ad.scale[e]) * ((x6[m] @ A6[e].t()) @ B6[e].t()))
    rms = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    st6 = 0.9 * s6 + rms(o6) * p6 * (1.2 * torch.tanh(g6))
    y6 = rms(st6) * n6
    ((y6 * dy.cpu().double()).sum() + (st6 * d_s.cpu().double()).sum()).backward()
    for name, got, ref in (("out", out, o6), ("y", y, y6), ("dx", dx, x6.grad), ("d_res", d_res, s6.grad), ("d_norm", d_norm, n6.grad),
                           ("d_post", d_post, p6.grad), ("d_gate", d_gate, g6.grad), ("dw1", dw1, W1.grad), ("dw2", dw2, W2.grad),
                           ("da", ad.da, A6.grad), ("db", ad.db, B6.grad)):
        err = oracle.max_norm_rel_err(got.detach().cpu().double().numpy(), ref.detach().numpy())
        assert err <= 3e-2, (name, err)

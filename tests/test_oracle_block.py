"""Pins of the block operators' oracle (no GPU): the norm's and the router's gradients against
torch.autograd on a float64 forward and against differences, the choice against torch.topk
where there is no tie, and ties, masks and groups on hand-worked rows."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block as ob


def test_round_bf16_matches_torch():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4096).astype(np.float32) * 3,
                        np.array([0.0, -0.0, 1.00390625, 1.01171875, 3.3e38, np.inf, -np.inf, np.nan], np.float32)])
    ref = torch.from_numpy(v).to(torch.bfloat16).float().numpy()
    assert np.array_equal(ob.round_bf16(v), ref, equal_nan=True)


def test_rmsnorm_and_gradients_match_autograd():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 24, generator=g).to(torch.bfloat16)
    res = torch.randn(5, 24, generator=g).to(torch.bfloat16)
    w = torch.randn(24, generator=g)
    s, rstd, y = ob.rmsnorm(x.float().numpy(), res.float().numpy(), w.numpy(), 1e-5)
    st = torch.from_numpy(s).double().requires_grad_(True)
    wt = w.double().requires_grad_(True)
    yt = st / torch.sqrt(st.square().mean(1, keepdim=True) + 1e-5) * wt
    # bf16 half step on y, fp32 products
    assert (np.abs(y - yt.detach().numpy()) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(yt.detach().numpy())).all()
    dy = torch.randn(5, 24, generator=g, dtype=torch.float64)
    yt.backward(dy)
    r64 = (1.0 / np.sqrt((s.astype(np.float64) ** 2).mean(1) + 1e-5))
    dx, dw = ob.rmsnorm_backward(dy.numpy(), s.astype(np.float64), w.double().numpy(), r64)
    assert np.abs(dx - st.grad.numpy()).max() < 1e-12 and np.abs(dw - wt.grad.numpy()).max() < 1e-12


def test_rmsnorm_gradient_matches_differences():
    rng = np.random.default_rng(2)
    s, w, dy = rng.standard_normal((2, 8)), rng.standard_normal(8), rng.standard_normal((2, 8))

    def f(s):
        return ((s / np.sqrt((s * s).mean(1, keepdims=True) + 1e-3) * w) * dy).sum()

    rstd = 1.0 / np.sqrt((s * s).mean(1) + 1e-3)
    dx, _ = ob.rmsnorm_backward(dy, s, w, rstd)
    for i in np.ndindex(2, 8):
        d = np.zeros((2, 8))
        d[i] = 1e-6
        assert abs((f(s + d) - f(s - d)) / 2e-6 - dx[i]) < 1e-7


CONFIGS = [dict(score=a, normalize=b, scale=c) for a in ("softmax", "sigmoid") for b in (True, False) for c in (1.0, 2.5)]


@pytest.mark.parametrize("kw", CONFIGS, ids=[f"{c['score']}-{c['normalize']}-{c['scale']}" for c in CONFIGS])
def test_router_gradient_matches_differences_and_autograd(kw):
    rng = np.random.default_rng(3)
    l, K = rng.standard_normal((4, 10)), 3
    idx, w = ob.router_topk(l, K, **kw)
    assert np.array_equal(idx, torch.from_numpy(l).topk(K, dim=1)[1].numpy())
    dw = rng.standard_normal((4, K))
    got = ob.router_topk_backward(dw, l, idx, **kw)
    lt = torch.from_numpy(l).requires_grad_(True)
    at = torch.from_numpy(idx)
    s = torch.softmax(lt, 1) if kw["score"] == "softmax" else torch.sigmoid(lt)
    wt = s.gather(1, at)
    wt = (wt / wt.sum(1, keepdim=True) if kw["normalize"] else wt) * kw["scale"]
    assert np.abs(wt.detach().numpy() - w).max() < 1e-14
    wt.backward(torch.from_numpy(dw))
    assert np.abs(lt.grad.numpy() - got).max() < 1e-13
    for i in np.ndindex(4, 10):
        d = np.zeros_like(l)
        d[i] = 1e-6
        v = [np.array([ob.chosen_weights(r, list(p), kw["score"], kw["normalize"]) for r, p in zip(l + q, idx)])
             for q in (d, -d)]
        assert abs(((v[0] - v[1]) * dw).sum() * kw["scale"] / 2e-6 - got[i]) < 1e-7


def test_router_ties_masks_and_groups_by_hand():
    inf = np.inf
    l = np.array([[1.0, 3.0, 3.0, 2.0],          # tie: the lower index first
                  [-inf, 5.0, np.nan, -inf],     # one expert left of two asked for
                  [-inf, -inf, -inf, -inf],      # none
                  [inf, 0.0, inf, -FLT]])        # infinities share, the lowest value is a number
    idx, w = ob.router_topk(l, 2)
    assert idx.tolist() == [[1, 2], [1, -1], [-1, -1], [0, 2]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0]
    assert w[3].tolist() == [0.5, 0.5]
    # groups {0,1}, {2,3}: one expert of 9 against two of 5: by the best, by the sum of two
    l = np.log(np.array([[9.0, 1.0, 6.0, 6.0]]))
    assert ob.router_topk(l, 2, groups=2, topk_groups=1, group_top=1)[0].tolist() == [[0, 1]]
    assert ob.router_topk(l, 2, groups=2, topk_groups=1, group_top=2)[0].tolist() == [[2, 3]]
    # the bias chooses, the weights are the scores'
    idx, w = ob.router_topk(np.zeros((1, 4)), 2, score="sigmoid", bias=np.array([0.0, 0.2, 0.1, -inf]))
    assert idx.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]]


FLT = ob.FLT_MAX


def test_decode_oracle_is_the_layers():
    """On MXFP4 inputs the few-token oracle equals the layer's oracle."""
    from synth import MoEConfig, make_inputs
    cfg = MoEConfig("dec", 4, 128, 128, 6, 1, 4, 2, 16, "mxfp4")
    inp = make_inputs(cfg, 5)
    ref = oracle.moe_layer(inp)
    got = ob.expert_ffn_decode(inp.x.float().numpy(), None, inp.topk_idx.numpy(), inp.topk_weights.numpy(),
                               *(t.view(torch.uint8).numpy() for t in (inp.w1, inp.w1_scale, inp.w2, inp.w2_scale)),
                               expert_begin=1)
    assert np.abs(got - ref.out).max() <= 1e-9 * np.abs(ref.out).max()

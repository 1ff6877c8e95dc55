"""The sigmoid router on tokens whose chosen logits are all strongly negative, against the float64 oracle: above -88 the
scores are fp32 numbers, but their reciprocal times a gradient need not be one; below, they are none, but the normalised weights, and the
gradients with them, are ratios of such scores and ordinary numbers. A score that is 0 in float64 (1 / (1 + e^-z) for z
below -709.78) is 0.

Tolerances as for the router in general: a weight is a ratio of scores, exp of an fp32 logit z (off by |z| 2^-24) with a few
roundings, over a sum of at most 16 of them: relative 2 (|z| + 16) 2^-24. A gradient is such a weight times a difference of
d_topk_weights * scale, at most twice their largest, and a sigmoid: four times that relative error of the largest term."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import block as ob

from _gpu import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


def gradient(l, idx, w, dw, cfg):
    """The gradient for the oracle's choice and weights, in the form that divides by no small sum."""
    d_logits = np.zeros(l.shape)
    for t in range(l.shape[0]):
        on = idx[t] >= 0
        at, p, d = idx[t][on], w[t][on] / cfg.scale, dw[t][on].astype(np.float64) * cfg.scale
        mean = (p * d).sum() if cfg.normalize else 0.0
        d_logits[t, at] = p * (d - mean) * (1.0 - ob.scores(l[t], "sigmoid")[at])
    return d_logits


@pytest.mark.parametrize("E,K", [(2, 2), (40, 8), (256, 16), (300, 3), (1024, 16)])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("size", [1.0, 1e2, 1e6])
def test_gradient_where_scores_are_small(E, K, normalize, size):
    say("router gradient of small scores", E, K, normalize, size)
    cfg = moe.RouterConfig(score="sigmoid", normalize=normalize, scale=2.5)
    g = torch.Generator().manual_seed(E + K)
    means = torch.tensor([-60.0, -80.0, -84.0, -85.5, -86.5])
    logits = means[:, None] + torch.rand(5, E, generator=g)
    dw = size * torch.randn(5, K, generator=g)
    l = logits.double().numpy()
    idx, w = ob.router_topk(l, K, score="sigmoid", normalize=normalize, scale=2.5)
    ref = gradient(l, idx, w, dw.numpy(), cfg)
    d = torch.full((5, E), 5.0, device="cuda")
    moe.moe_router_topk_backward(dw.cuda(), logits.cuda(), torch.from_numpy(idx).int().cuda(), d, cfg)
    torch.cuda.synchronize()
    lead = np.zeros((5, E))
    np.put_along_axis(lead, idx, w / 2.5, 1)
    tol = 8 * 2 * (87 + 16) * U * np.abs(dw.numpy()).max(1, keepdims=True) * 2.5 * lead + 2.0 ** -120 * size
    assert (np.abs(d.double().cpu().numpy() - ref) <= tol).all()


def far_rows(E, seed):
    """Rows of E logits: all of them around one far place, spread over several, and masked ones among them."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for mean in (-60.0, -80.0, -86.0, -88.0, -88.7, -89.0, -90.0, -100.0, -103.0, -104.5, -120.0, -300.0, -700.0):
        rows.append(mean + torch.rand(E, generator=g))
        rows.append(torch.full((E,), mean))
    rows.append(-80 - 40 * torch.rand(E, generator=g))
    rows.append(-709 * torch.rand(E, generator=g))
    rows.append(torch.full((E,), -710.0))                       # 0 in float64
    rows.append(-705 - 10 * torch.rand(E, generator=g))         # some are
    r = torch.full((E,), -INF)
    r[: (E + 1) // 2] = -95.0
    rows.append(r)                                              # switched off, not far
    r = torch.full((E,), -100.0)
    r[0] = 3.0
    rows.append(r)                                              # one that is not far
    r = torch.full((E,), -100.0)
    r[-1] = -60.0
    rows.append(r)
    return torch.stack(rows)


def expected(l, K, cfg, bias, dw):
    idx, w = ob.router_topk(l, K, bias=bias, score=cfg.score, normalize=cfg.normalize, scale=cfg.scale)
    return idx, w, gradient(l, idx, w, dw, cfg)


@pytest.mark.parametrize("E,K,many", [(4, 1, False), (4, 2, False), (40, 8, False), (128, 8, True), (256, 16, True), (300, 16, False),
                                      (1024, 6, False)])
@pytest.mark.parametrize("normalize,scale", [(True, 1.0), (True, 2.5), (False, 2.5)])
@pytest.mark.parametrize("size", [1.0, 1e4])
def test_far_logits(E, K, many, normalize, scale, size):
    say("router far", E, K, many, normalize, scale, size)
    cfg = moe.RouterConfig(score="sigmoid", normalize=normalize, scale=scale)
    for dt, with_bias in ((torch.float32, False), (torch.float32, True), (torch.bfloat16, False)):
        rows = far_rows(E, E + K).to(dt)
        n = rows.shape[0]
        g = torch.Generator().manual_seed(7)
        bias = 0.3 * torch.randn(E, generator=g) if with_bias else None
        dw = size * torch.randn(n, K, generator=g)
        l = rows.double().numpy()
        ref_i, ref_w, ref_d = expected(l, K, cfg, None if bias is None else bias.numpy(), dw.numpy())
        # more than 4096 tokens: another layout of the forward pass
        at = torch.arange(4097 if many else n) % n
        idx = torch.empty(len(at), K, dtype=torch.int32, device="cuda")
        w = torch.empty(len(at), K, device="cuda")
        logits = rows[at].cuda()
        moe.moe_router_topk(logits, idx, w, cfg, bias=None if bias is None else bias.cuda())
        d = torch.full_like(logits, 5.0)
        moe.moe_router_topk_backward(dw[at].cuda(), logits, idx, d, cfg)
        torch.cuda.synchronize()
        assert np.array_equal(idx.cpu().numpy(), ref_i[at])
        rel = 2 * (np.abs(np.where(np.isfinite(l), l, 0.0)).max(1, keepdims=True) + 16) * U
        assert (np.abs(w.cpu().numpy() - ref_w[at]) <= (rel * ref_w + 2.0 ** -126)[at]).all()
        lead = np.zeros((n, E))                                 # the weight of the chosen
        for t in range(n):
            lead[t, ref_i[t][ref_i[t] >= 0]] = ref_w[t][ref_i[t] >= 0] / scale
        big = np.abs(dw.numpy()).max(1, keepdims=True) * scale
        half = 2.0 ** -8 * np.abs(ref_d) if dt == torch.bfloat16 else 0.0
        tol = 4 * rel * 2 * big * lead + half + 2.0 ** -120 * max(1.0, size)
        assert (np.abs(d.double().cpu().numpy() - ref_d[at]) <= tol[at]).all()


def test_known_ratios():
    """(-90, -91): 2.5 / (1 + e^-1) and the rest; four of -100: a quarter of 2.5 each; none above float64's range: 0."""
    say("router far ratios")
    cfg = moe.RouterConfig(score="sigmoid", scale=2.5)
    l = torch.tensor([[-90.0, -91.0], [-88.5, -88.5], [-710.0, -711.0]], device="cuda")
    idx, w = torch.empty(3, 2, dtype=torch.int32, device="cuda"), torch.empty(3, 2, device="cuda")
    d, dw = torch.empty_like(l), torch.tensor([[1.0, -1.0]] * 3, device="cuda")
    moe.moe_router_topk(l, idx, w, cfg)
    moe.moe_router_topk_backward(dw, l, idx, d, cfg)
    torch.cuda.synchronize()
    p = 1.0 / (1.0 + np.exp(-1.0))
    assert np.allclose(w.cpu().numpy(), [[2.5 * p, 2.5 * (1 - p)], [1.25, 1.25], [0.0, 0.0]], rtol=2e-5, atol=0)
    assert np.allclose(d.cpu().numpy(), [[5 * p * (1 - p), -5 * p * (1 - p)], [1.25, -1.25], [0.0, 0.0]], rtol=4e-5, atol=0)

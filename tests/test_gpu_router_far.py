"""The sigmoid router's gradient on tokens whose chosen logits are all strongly negative, against the float64 oracle: above -88 the
scores are fp32 numbers, but their reciprocal times a gradient need not be one.

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

"""The router's choice and its backward pass on the GPU against the float64 oracle.

The indices are equal, always. Weights are fp32: exp of a difference d of two fp32 logits is off by
|d| 2^-24 (the difference's rounding) and a few units, sums of at most 1024 positive terms by 11
roundings, one division, one product: relative 2 (|d| + 16) 2^-24 in all, and what lies below fp32's
normal range absolutely 2^-126. Gradients are products of such weights with differences of
d_topk_weights: the same relative error of the largest term in play."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import block as ob

from _gpu import say

pytestmark = pytest.mark.gpu

INF = float("inf")
U = 2.0 ** -24


def run(logits, K, cfg, bias=None):
    l = logits.cuda()
    T = l.shape[0]
    idx = torch.full((T, K), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), 77.0, device="cuda")
    moe.moe_router_topk(l, idx, w, cfg, bias=None if bias is None else bias.cuda())
    torch.cuda.synchronize()
    return idx, w


def oracle_kw(cfg):
    return dict(score=cfg.score, normalize=cfg.normalize, groups=cfg.groups, topk_groups=cfg.topk_groups,
                group_top=cfg.group_top, scale=float(np.float32(cfg.scale)))


def spread(l):
    """The largest difference of two finite logits, per token."""
    f = np.where(np.isfinite(l) & (np.abs(l) < 1e30), l, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            d = np.nanmax(f, 1) - np.nanmin(f, 1)
    return np.where(np.isnan(d), 0.0, np.maximum(d, np.nan_to_num(np.nanmax(np.abs(f), 1, initial=0.0))))


def check(logits, K, cfg, bias=None):
    l = logits.float().numpy().astype(np.float64)
    ref_i, ref_w = ob.router_topk(l, K, bias=None if bias is None else bias.numpy(), **oracle_kw(cfg))
    idx, w = run(logits, K, cfg, bias)
    assert np.array_equal(idx.cpu().numpy(), ref_i)
    rel = (2 * (spread(l) + 16) * U)[:, None]
    assert (np.abs(w.cpu().numpy() - ref_w) <= rel * np.abs(ref_w) + 2.0 ** -126).all()
    # backward
    g = torch.Generator().manual_seed(K)
    dw = torch.randn(l.shape[0], K, generator=g)
    dl = torch.full_like(logits, 5.0).cuda()
    moe.moe_router_topk_backward(dw.cuda(), logits.cuda(), idx, dl, cfg)
    torch.cuda.synchronize()
    ref = ob.router_topk_backward(dw.numpy(), l, ref_i, **oracle_kw(cfg))
    got = dl.float().cpu().numpy().astype(np.float64)
    s = np.stack([ob.scores(r, cfg.score) for r in l])
    # the terms of a token: scores (or weights) times d, d at most max|dw| * scale
    big = np.abs(dw.numpy()).max(1, keepdims=True) * abs(cfg.scale)
    lead = np.zeros_like(s)
    for t in range(l.shape[0]):
        at = [e for e in ref_i[t] if e >= 0]
        if at:
            w_t = ob.chosen_weights(l[t], at, cfg.score, cfg.normalize)
            lead[t, at] = w_t
            if cfg.score == "softmax" and not cfg.normalize:
                lead[t] = np.maximum(lead[t], s[t])
    tol = 4 * rel * 2 * big * lead + (2.0 ** -8 * np.abs(ref) if logits.dtype == torch.bfloat16 else 0) + 2.0 ** -120
    assert (np.abs(got - ref) <= tol).all()
    return idx, w


ALL = [moe.RouterConfig(score=a, normalize=b, scale=c) for a in ("softmax", "sigmoid") for b, c in ((True, 1.0), (False, 2.5))]
ids = lambda c: f"{c.score}-{c.normalize}-{c.groups}.{c.topk_groups}.{c.group_top}"  # noqa: E731


# every register layout, smallest, odd and largest
@pytest.mark.parametrize("E", [1, 2, 7, 16, 64, 65, 128, 129, 256, 257, 512, 513, 1000, 1024])
@pytest.mark.parametrize("cfg", ALL, ids=ids)
def test_every_width(E, cfg):
    say("router", E, cfg)
    g = torch.Generator().manual_seed(E)
    for T, K, dt in ((1, min(E, 8), torch.float32), (9, min(E, 16), torch.bfloat16), (6, 1, torch.float32)):
        check(2 * torch.randn(T, E, generator=g).to(dt), K, cfg)


@pytest.mark.parametrize("E", [8, 72, 128, 256, 384, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias(E, score):
    say("router bias", E, score)
    g = torch.Generator().manual_seed(E + 1)
    l = torch.randn(13, E, generator=g)
    b = 0.3 * torch.randn(E, generator=g)
    b[3], b[5] = -INF, float("nan")
    check(l, min(8, E - 2), moe.RouterConfig(score=score), b)
    check(l.to(torch.bfloat16), 3, moe.RouterConfig(score=score, normalize=False), b)


GROUPS = [(64, 8, 3, 1), (64, 8, 3, 2), (256, 8, 4, 2), (160, 8, 3, 1), (60, 60, 20, 2), (64, 64, 16, 1), (1024, 64, 9, 2),
          (96, 32, 8, 2), (48, 16, 5, 2), (66, 22, 7, 1), (1000, 4, 2, 2), (32, 16, 16, 1)]


@pytest.mark.parametrize("E,G,keep,top", GROUPS)
@pytest.mark.parametrize("score,with_bias", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_groups(E, G, keep, top, score, with_bias):
    say("router groups", E, G, keep, top, score, with_bias)
    g = torch.Generator().manual_seed(E + G)
    l = torch.randn(11, E, generator=g)
    l[2] = -INF
    l[3, E // G:] = -INF                         # one group left
    l[4, torch.rand(E, generator=g) < 0.7] = -INF
    b = 0.1 * torch.randn(E, generator=g) if with_bias else None
    check(l, min(8, keep * (E // G)), moe.RouterConfig(score=score, groups=G, topk_groups=keep, group_top=top, scale=2.5), b)


@pytest.mark.parametrize("cfg", ALL + [moe.RouterConfig(groups=4, topk_groups=2, group_top=2)], ids=ids)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_ties_masks_and_infinities(cfg, dt):
    say("router masks", cfg, dt)
    E, K = 16, 6
    low = torch.finfo(dt).min
    rows = [torch.zeros(E), torch.full((E,), -INF), torch.full((E,), low), torch.full((E,), float("nan")),
            torch.full((E,), INF), torch.arange(E) // 3 * 1.0, -torch.arange(E) // 5 * 1.0]
    r = torch.full((E,), -INF)
    r[9] = 1.0
    rows.append(r)                               # one expert
    r = torch.full((E,), low)
    r[4:7] = torch.tensor([0.5, float("nan"), 0.5])
    rows.append(r)                               # the type's lowest value as a mask
    r = torch.arange(E) * 1.0
    r[[2, 7, 15]] = torch.tensor([INF, -INF, INF])
    rows.append(r)
    r = torch.zeros(E)
    r[::2] = -0.0
    rows.append(r)                               # zeros of both signs are a tie
    rows.append(torch.linspace(-200, 90, E))
    check(torch.stack(rows).to(dt), K, cfg)


def test_close_scores_are_told_apart():
    """Scores + bias that a 32-bit sum would tie or swap: sigmoid near 1, bias differences of 2^-26."""
    say("router close")
    E = 32
    l = torch.full((1, E), 12.0)
    l[0] += torch.arange(E) * 1e-5
    b = torch.arange(E - 1, -1, -1).float() * 2.0 ** -32
    check(l, 8, moe.RouterConfig(score="sigmoid"), b)
    check(l, 8, moe.RouterConfig(score="softmax"), b)


def hard_rows(E, dt, seed):
    """Rows whose order hangs on a key's last bits: clusters a few units apart, exact ties, both, around any
    place of the choice, masked or not."""
    g = torch.Generator().manual_seed(seed)
    rows = [torch.randn(E, generator=g), torch.zeros(E), torch.randn(E, generator=g).sign()]
    for unit in (2.0 ** -23, 2.0 ** -20, 2.0 ** -16):
        steps = torch.randint(0, 40, (4, E), generator=g).float()
        rows += list(1.0 + steps * unit)                                     # one cluster
        rows += list(torch.randint(0, 3, (4, E), generator=g).float() + steps * unit)
    for i in range(3, len(rows), 3):
        rows[i] = torch.where(torch.rand(E, generator=g) < 0.4, torch.tensor(-INF), rows[i])
    return torch.stack(rows).to(dt)


HARD = [moe.RouterConfig(), moe.RouterConfig(score="sigmoid", normalize=False), moe.RouterConfig(groups=4, topk_groups=2),
        moe.RouterConfig(score="sigmoid", groups=8, topk_groups=3, group_top=2, scale=2.5),
        moe.RouterConfig(score="softmax", groups=4, topk_groups=3, group_top=2)]


@pytest.mark.parametrize("E", [16, 64, 72, 128, 200, 256, 512, 1024])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_close_keys(E, dt):
    """The kernels choose by shortened keys first: every way that can end, one token a wave."""
    say("router close keys", E, dt)
    rows = hard_rows(E, dt, E)
    bias = 2.0 ** -22 * torch.randint(-4, 4, (E,), generator=torch.Generator().manual_seed(E)).float()
    for cfg in HARD:
        K = min(8, cfg.topk_groups * (E // cfg.groups))
        for k in (1, K):
            check(rows, k, cfg)
        check(rows, K, cfg, bias)


@pytest.mark.parametrize("E", [16, 60, 64, 72, 128, 200, 256])
@pytest.mark.parametrize("cfg", HARD, ids=ids)
def test_four_tokens_a_wave(E, cfg):
    """More than 4096 tokens take another layout: the same rows again and again, an odd number."""
    say("router many", E, cfg)
    if E % cfg.groups:
        E += cfg.groups - E % cfg.groups
    for dt, with_bias in ((torch.float32, False), (torch.float32, True), (torch.bfloat16, False)):
        rows = hard_rows(E, dt, E + 1)
        bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)) if with_bias else None
        n, T = rows.shape[0], 4097 + 30
        for K in {1, min(8, cfg.topk_groups * (E // cfg.groups)), min(16, cfg.topk_groups * (E // cfg.groups))}:
            few, few_w = check(rows, K, cfg, bias)
            at = (torch.arange(T) * 5) % n
            idx, w = run(rows[at], K, cfg, bias)
            assert torch.equal(idx, few[at.cuda()])
            assert (w - few_w[at.cuda()]).abs().max() <= 2.0 ** -20 * cfg.scale      # sums in another order
            dw = torch.randn(n, K, generator=torch.Generator().manual_seed(1))[at].contiguous().cuda()
            dl, ref = torch.empty(T, E, dtype=dt, device="cuda"), torch.empty(n, E, dtype=dt, device="cuda")
            moe.moe_router_topk_backward(dw, rows[at].cuda(), idx, dl, cfg)
            first = torch.tensor([int((at == i).nonzero()[0]) for i in range(n)])
            moe.moe_router_topk_backward(dw[first.cuda()].contiguous(), rows.cuda(), few, ref, cfg)
            torch.cuda.synchronize()
            assert torch.equal(dl, ref[at.cuda()])


def test_many_tokens_match_few():
    say("router many tokens")
    for E, K, cfg in ((24, 4, moe.RouterConfig()), (130, 8, moe.RouterConfig(score="sigmoid"))):
        T = 300_003 if E < 64 else 70_001
        g = torch.Generator(device="cuda").manual_seed(E)
        l = torch.randn(T, E, generator=g, device="cuda")
        idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
        w = torch.empty(T, K, device="cuda")
        moe.moe_router_topk(l, idx, w, cfg)
        top, at = l.topk(K, dim=1)
        assert torch.equal(idx.long(), at)
        dw, dl = torch.randn(T, K, generator=g, device="cuda"), torch.empty_like(l)
        moe.moe_router_topk_backward(dw, l, idx, dl, cfg)
        pick = torch.tensor([0, 3, 65535, 65536, T - 1], device="cuda")
        dl2 = torch.empty_like(l[pick])
        moe.moe_router_topk_backward(dw[pick].contiguous(), l[pick].contiguous(), idx[pick].contiguous(), dl2, cfg)
        torch.cuda.synchronize()
        assert torch.equal(dl[pick], dl2)


def test_backward_takes_foreign_indices():
    """Places of no expert, of switched-off experts and doubled ones; in place of the logits."""
    say("router backward foreign")
    l = torch.randn(4, 12, generator=torch.Generator().manual_seed(0))
    l[1, 3] = -INF
    idx = torch.tensor([[0, -1, 5], [3, 2, 12], [7, 7, 1], [-1, -1, -1]], dtype=torch.int32)
    dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(1))
    dw[0, 1] = float("nan")
    dw[3] = float("nan")
    for cfg in ALL:
        d = l.clone().cuda()
        moe.moe_router_topk_backward(dw.cuda(), d, idx.cuda(), d, cfg)
        torch.cuda.synchronize()
        ref = ob.router_topk_backward(torch.nan_to_num(dw).numpy(), l.double().numpy(), idx.numpy(), **oracle_kw(cfg))
        assert np.abs(d.cpu().numpy() - ref).max() <= 64 * U * max(1.0, dw[~dw.isnan()].abs().max().item()) * cfg.scale * 4


def test_no_tokens_and_refusals():
    say("router refusals")
    e = torch.empty(0, 8, device="cuda")
    moe.moe_router_topk(e, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    l, i, w = torch.zeros(3, 8, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    for bad in ((l.half(), i, w), (l, i.long(), w), (l, i, w[:2]), (l, i, w.bfloat16()), (l[0], i, w), (l.t(), i, w)):
        with pytest.raises(ValueError):
            moe.moe_router_topk(*bad)
    with pytest.raises(ValueError):
        moe.moe_router_topk(l, i, w, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_router_topk_backward(w, l, i, l.bfloat16())
    with pytest.raises(moe.MoeError):
        moe.moe_router_topk(l, i, w, moe.RouterConfig(groups=3))

"""Infinities in the adapters' products: where 32-bit numbers give an infinity, so do the kernels, with its sign, however v and dv
enter the products; where they give NaN (infinities of both signs, 0 times infinity), NaN; and nothing else changes."""
import numpy as np
import pytest
import torch

import test_gpu_adapter as ad

from _gpu import say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF = float("inf")


def make(T, n, K, N, R, seed=0):
    d = ad.make(T, n, K, N, R, seed, ids=[t % n for t in range(T)])
    # some v and dv are whole bf16 numbers: no bits are left for a second part
    d["x"][::3] = 0
    d["x"][::3, 0] = 1
    d["dout"][::3] = 0
    d["dout"][::3, 0] = 1
    return d


def plan_of(d, tile):
    return None if tile is None else ad.make_plan(d, tile)


SIZES = [(40, 3, 64, 136, 24, None), (64, 2, 264, 520, 64, None), (300, 3, 136, 264, 16, 16), (400, 2, 136, 264, 40, 128), (600, 2, 264, 136, 64, 128),
         (600, 2, 136, 264, 128, 128), (300, 2, 136, 72, 256, 128), (300, 2, 72, 136, 256, 16)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_b(size, sign):
    say("infinite b", size, sign)
    T, n, K, N, R, tile = size
    d = make(T, n, K, N, R)
    ref = ad.forward(d, plan_of(d, tile))
    d["b"][1, 5, 2] = sign * INF
    d["b"][1, 70, 0] = -sign * INF
    o = ad.forward(d, plan_of(d, tile))
    rows = (d["ids"] == 1).nonzero().squeeze(1)
    v = o["v"][rows]
    assert (v[:, [0, 2]] != 0).all()
    for col, r, s in ((5, 2, sign), (70, 0, -sign)):
        assert torch.equal(o["out"][rows, col].float(), s * INF * torch.sign(v[:, r])), col
    keep = torch.ones(T, N, dtype=torch.bool, device="cuda")
    for col in (5, 70):
        keep[rows, col] = False
    assert torch.equal(o["out"][keep], ref["out"][keep]) and torch.equal(o["v"], ref["v"])
    d["b"][1, 5, 3] = INF                         # two of them, of one sign or of two
    out = ad.forward(d, plan_of(d, tile))["out"][rows, 5].float()
    assert torch.equal(torch.isnan(out), torch.sign(v[:, 2]) * sign != torch.sign(v[:, 3]))


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_infinite_and_zero_v(size):
    """x of 0: v is 0, and 0 times infinity NaN. An infinite x: v is, and out by the signs of b."""
    say("infinite v", size)
    T, n, K, N, R, tile = size
    d = make(T, n, K, N, R)
    d["x"][1] = 0
    d["x"][1 + n, 3] = INF
    d["b"][1, 5, 2] = INF
    d["b"][1, 6, 2] = 0
    d["a"][1, :, 3] = 0.5
    o = ad.forward(d, plan_of(d, tile))
    assert torch.isnan(o["out"][1, 5]) and torch.isfinite(o["out"][1, 6])
    assert (o["v"][1 + n] == INF).all()
    b = d["b"][1].float()
    want = torch.where((b != 0).all(1) & ((b > 0).all(1) | (b < 0).all(1)), torch.sign(b[:, 0]) * INF, torch.full_like(b[:, 0], float("nan")))
    assert torch.equal(torch.isnan(o["out"][1 + n]), torch.isnan(want))
    d["b"][1] = d["b"][1].abs() + 0.25            # all of one sign, an infinite one among them
    d["b"][1, 5, 2] = INF
    assert (ad.forward(d, plan_of(d, tile))["out"][1 + n] == INF).all()


@pytest.mark.parametrize("size", [s for s in SIZES if s[5]] + [(40, 3, 64, 136, 24, 16), (2100, 1, 136, 136, 16, 32)], ids=str)
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_values_in_the_backward_pass(size, sign):
    say("infinite backward", size, sign)
    T, n, K, N, R, tile = size
    d = make(T, n, K, N, R)
    e = n - 1
    plan = ad.make_plan(d, tile)
    o = ad.forward(d, plan)
    ref = ad.backward(d, o, plan)
    # an infinite a: dx of its column
    bad = dict(d, a=d["a"].clone())
    bad["a"][e, 2, 6] = sign * INF
    g = ad.backward(bad, o, plan)
    rows = (d["ids"] == e).nonzero().squeeze(1)
    # dv of that rank, by its own products: da of a column of ones
    dv = ad.backward(dict(d, a=torch.eye(R, K, device="cuda").to(BF16).expand(n, R, K).contiguous()), o, plan, want=("dx",), base=False)["dx"] if K >= R else None
    got = g["dx"][rows, 6].float()
    if dv is not None:
        s = torch.sign(dv[rows, 2].float())
        on = s != 0
        assert on.any() and torch.equal(got[on], s[on] * sign * INF)
    assert not torch.isnan(got).any() and torch.isinf(got).all()
    keep = torch.ones(T, K, dtype=torch.bool, device="cuda")
    keep[rows, 6] = False
    assert torch.equal(g["dx"][keep], ref["dx"][keep]) and torch.equal(g["da"], ref["da"]) and torch.equal(g["db"], ref["db"])
    # an infinite dout: db of its column by the signs of v
    for t in (int(rows[0]), int(rows[1])):
        bad = dict(d, dout=d["dout"].clone())
        bad["dout"][t, 9] = sign * INF
        g = ad.backward(bad, o, plan, want=("db",))
        assert (o["v"][t] != 0).all()
        assert torch.equal(g["db"][e, 9], torch.sign(o["v"][t]) * sign * INF)
        keep = torch.ones(n, N, R, dtype=torch.bool, device="cuda")
        keep[e, 9] = False
        assert torch.equal(g["db"][keep], ref["db"][keep])
    # an infinite x: da of its column by the signs of dv
    t = int(rows[0])
    bad = dict(d, x=d["x"].clone())
    bad["x"][t, 4] = sign * INF
    g = ad.backward(bad, o, plan, want=("da",))
    assert not torch.isnan(g["da"]).any() and torch.isinf(g["da"][e, :, 4]).all()
    if dv is not None:
        s = torch.sign(dv[t, :R].float())
        assert torch.equal(g["da"][e, s != 0, 4], s[s != 0] * sign * INF)
    keep = torch.ones(n, R, K, dtype=torch.bool, device="cuda")
    keep[e, :, 4] = False
    assert torch.equal(g["da"][keep], ref["da"][keep])


@pytest.mark.parametrize("tile", [None, 128])
def test_largest_finite_v(tile):
    """v that a bf16 rounding would make infinite: x 2^127 times 1 + 255/256 and more."""
    T, n, K, N, R = (8, 1, 16, 64, 8) if tile is None else (300, 1, 16, 64, 8)
    d = ad.make(T, n, K, N, R, ids=[0] * T)
    d["x"].zero_(), d["a"].zero_(), d["b"].fill_(0), d["base"].zero_()
    d["scale"] = torch.ones(1, device="cuda")
    d["x"][:, 0], d["x"][:, 1] = 2.0 ** 127, 2.0 ** 127
    d["a"][0, 0, 0], d["a"][0, 0, 1] = 1 + 127 / 128, 2.0 ** -8 * (1 + 127 / 128)
    d["b"][0, 0, 0] = 0.5
    o = ad.forward(d, plan_of(d, tile))
    v = 2.0 ** 127 * ((1 + 127 / 128) * (1 + 2.0 ** -8))
    assert np.float32(v) < np.finfo(np.float32).max and (o["v"][:, 0].double() == float(np.float32(v))).all()
    out = o["out"][:, 0].double()
    assert torch.isfinite(out).all() and (out - v / 2).abs().max() <= 2.0 ** -8 * v / 2 and (o["out"][:, 1:] == 0).all()

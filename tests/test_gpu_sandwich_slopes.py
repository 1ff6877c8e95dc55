"""The gates' gradients far out in the tails of sigmoid and tanh, where f (1 - f) and 1 - f^2 would cancel.

Without norms d_gate = branch_scale act'(gate) d_s x of each value, of positive d_s and x so that nothing cancels in sums. With e = exp(-|z|) (u =
exp(-2 |z|)) the slope is e / (1 + e)^2 (4 u / (1 + u)^2): in units of U = 2^-24 the exponential is off by 4 (2 units in the last
place), the reciprocal of the rounded 1 + e by 3, its square by 6 and both products by 2: 12 U relative, and d_gate's three products
3 more. A row's sum adds at most 80 U (53 terms in a chain, the terms' own roundings), a column's T + 24. Slopes below e^-87 may be
taken as 0: at most 2^-124 of the rest."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import test_gpu_sandwich as sw
from oracle import behind as ob

from _gpu import say

pytestmark = pytest.mark.gpu

U, HALF = sw.U, sw.HALF
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
FAR = 2.0 ** -124


def bare(T, H, gate, gdt, seed=1):
    """No norms; gates over the whole range of the activations, both signs."""
    g = torch.Generator().manual_seed(seed)
    d = dict(x=torch.rand(T, H, generator=g).add(0.5).to(BF16), d_s=torch.rand(T, H, generator=g).add(0.5).to(BF16),
             gate=(torch.rand(*sw.SHAPE[gate](T, H), generator=g) * 240 - 120).to(gdt))
    # as many within the range where the activations bend
    z = d["gate"].flatten()
    z[::2] = (z[::2].float() / 8).to(gdt)
    d = {k: v.cuda() for k, v in d.items()}
    return dict(d, res=None, wp=None, w=None, dy=None)


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
@pytest.mark.parametrize("gdt", [F32, BF16])
def test_slopes_of_saturated_gates(act, gate, gdt):
    for T, H in ((300, 8), (37, 520), (19, 1032), (130, 4104), (5, 8200), (3, 16392)):
        say("slopes", act, gate, gdt, T, H)
        d = bare(T, H, gate, gdt)
        g = sw.backward(d, dict(s=None, r1=None, r2=None), act, 1.0, 0.75)
        x, d_s, z = (sw.f64(d[k]) for k in ("x", "d_s", "gate"))
        p = x * d_s * 0.75
        ref = ob.gate_slope(z, act) * p
        if gate == "row":
            ref, p, off = ref.sum(1, keepdims=True), p.sum(1, keepdims=True), 15 + 80
        elif gate == "channel":
            ref, p, off = ref.sum(0), p.sum(0), 15 + T + 24
        else:
            off = 15
        half = HALF if g["d_gate"].dtype == BF16 else U
        bad = np.abs(sw.f64(g["d_gate"]) - ref) > off * U * (1 + half) * ref + half * ref + FAR * p
        assert not bad.any(), (T, H, int(bad.sum()), (np.broadcast_to(z, ref.shape) if gate != "row" else z)[bad][:4],
                               sw.f64(g["d_gate"])[bad][:4], ref[bad][:4])
        # the factor itself there: d_x = branch_scale f d_s, f within 8 U
        f = ob.gate_act(z, act)
        dx = 0.75 * f * d_s
        assert (np.abs(sw.f64(g["dx"]) - dx) <= 12 * U * np.abs(dx) + HALF * np.abs(dx) + FAR * d_s).all()


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
def test_far_gates_with_norms(act, gate):
    for T, H, gdt in ((37, 520, BF16), (130, 1032, F32), (70, 7168, F32), (3, 16392, BF16)):
        say("far gates", act, gate, T, H)
        d = sw.make(T, H, T, gate=gate, gdt=gdt)
        d["gate"] *= 30
        o = sw.forward(d, act, 0.7, 1.3)
        sw.check_backward(d, o, sw.backward(d, o, act, 0.7, 1.3), act, 0.7, 1.3)


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("gdt", [F32, BF16])
def test_gates_that_are_not_finite(act, gdt):
    """An infinite gate has its factor's limit and no slope; NaN spoils its value, with a post-norm its row."""
    for T, H in ((6, 264), (6, 7168), (6, 8200)):
        say("gates not finite", act, gdt, T, H)
        for gate in ("row", "channel", "full"):
            d = bare(T, H, gate, gdt)
            flat = d["gate"].view(-1)
            flat[0], flat[1], flat[2] = INF, -INF, NAN
            z = sw.f64(d["gate"])
            g = sw.backward(d, dict(s=None, r1=None, r2=None), act)
            got, dx = sw.f64(g["d_gate"]).reshape(-1), sw.f64(g["dx"])
            assert got[0] == 0 and got[1] == 0 and np.isnan(got[2]) and np.isfinite(got[3:]).all()
            want = ob.gate_act(z, act) * sw.f64(d["d_s"])
            assert np.array_equal(np.isnan(dx), np.isnan(want))
            on = ~np.isnan(want)
            assert (np.abs(dx - want)[on] <= 16 * U * np.abs(want[on]) + HALF * np.abs(want[on]) + FAR * 2).all()
        d = sw.make(T, H, 5, gate="full", gdt=gdt)
        d["gate"][1, 3], d["gate"][4, 7], d["gate"][2, 5] = INF, -INF, NAN
        o = sw.forward(d, act)
        g = sw.backward(d, o, act)
        ok = torch.tensor([0, 1, 3, 4, 5], device="cuda")
        assert torch.isnan(g["dx"][2].float()).any() and torch.isfinite(g["dx"][ok].float()).all()
        assert g["d_gate"][1, 3] == 0 and g["d_gate"][4, 7] == 0 and torch.isfinite(g["d_gate"][ok].float()).all()

"""The forward pass with an activation, as exact as its roundings are counted. In units of U = 2^-24: the factor is off by 6 (expf 2 units
in the last place, 1 + e and the quotient half a unit each; tanhf 4), its scale adds 1, p has 3 (post_rstd and two products), p f
and the sum 1 each: within 16 U of the terms' magnitudes before the stream's bf16 half step."""
import numpy as np
import pytest

import test_gpu_sandwich as sw
from oracle import behind as ob

from _gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
@pytest.mark.parametrize("T,H", [(7, 520), (33, 4096), (19, 7168), (3, 32768)])
def test_stream_within_counted_roundings(act, gate, T, H):
    say("stream", act, gate, T, H)
    for spread, rs, bs in ((1.0, 1.0, 0.22), (30.0, 0.5, 1.5)):
        d = sw.make(T, H, T, gate=gate, gdt=sw.F32)
        d["gate"] *= spread
        o = sw.forward(d, act, rs, bs)
        x, res, wp, z = (sw.f64(d[k]) for k in ("x", "res", "wp", "gate"))
        rs32, bs32 = float(np.float32(rs)), float(np.float32(bs))
        s, _, p = ob.sandwich(x, res, wp, z, act, rs32, bs32, 1e-5)
        terms = np.abs(p * ob.gate_act(z, act) * bs32) + np.abs(res * rs32)
        assert (np.abs(sw.f64(o["s"]) - s) <= sw.HALF * np.abs(s) + 16 * sw.U * terms + 1e-37).all()

"""moe_sandwich_norm and its backward refuse bad arguments before anything is enqueued (no call here
reaches a launch), and the oracle's gradients are the derivatives of its forward pass. No GPU."""
import ctypes
import os

import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from combine_moe_dispatch_02_amd import _abi
from oracle import behind as ob

OK, INVALID, UNSUPPORTED = _abi.MOE_OK, _abi.MOE_ERR_INVALID, _abi.MOE_ERR_UNSUPPORTED
A = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(24)]     # never dereferenced
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40
CFG = dict(post_eps=1e-6, eps=1e-6, res_scale=1.0, branch_scale=1.0, gate=1, gate_act=1, gate_dtype=0)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        pytest.fail("libmoe355.so is not built (run __graft_entry__.build())")
    return _abi.load()


def cfg(**kw):
    return _abi.SandwichConfigT(*{**CFG, **kw}.values())


def fwd(lib, c=None, **kw):
    a = dict(x=A[0], res=A[1], wp=A[2], w=A[3], wt=0, gate=A[4], T=4, H=128, s=A[5], y=A[6], r1=A[7], r2=A[8], qd=0, q=None, qs=None)
    a.update(kw)
    c = cfg(**(c or {})) if c != "null" else None
    return lib.moe_sandwich_norm(a["x"], a["res"], a["wp"], a["w"], a["wt"], a["gate"], c, a["T"], a["H"], a["s"], a["y"], a["r1"],
                                 a["r2"], a["qd"], a["q"], a["qs"], None)


def bwd(lib, c=None, **kw):
    a = dict(dy=A[0], ds=A[1], x=A[2], s=A[3], wp=A[4], w=A[5], wt=0, gate=A[6], r1=A[7], r2=A[8], T=4, H=128, dx=A[9], dres=A[10],
             dw=A[11], dwp=A[12], dg=A[13], ws=A[14], n=BIG)
    a.update(kw)
    c = cfg(**(c or {})) if c != "null" else None
    return lib.moe_sandwich_norm_backward(a["dy"], a["ds"], a["x"], a["s"], a["wp"], a["w"], a["wt"], a["gate"], c, a["r1"], a["r2"],
                                          a["T"], a["H"], a["dx"], a["dres"], a["dw"], a["dwp"], a["dg"], a["ws"], a["n"], None)


NAN, INF = float("nan"), float("inf")
BAD_CFG = [dict(eps=-1.0), dict(eps=NAN), dict(post_eps=INF), dict(res_scale=NAN), dict(branch_scale=INF), dict(gate=-1), dict(gate=4),
           dict(gate_act=3), dict(gate_act=-1), dict(gate_dtype=2), dict(gate=0)]


@pytest.mark.parametrize("c", BAD_CFG, ids=str)
def test_config_refused(lib, c):
    assert fwd(lib, c) == INVALID and bwd(lib, c) == INVALID


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(s=None), dict(y=None), dict(T=-1), dict(H=0), dict(H=7), dict(wt=7), dict(qd=9), dict(q=A[9]), dict(qs=A[9]),
    dict(qd=1, q=A[9]), dict(qd=2, qs=A[9]), dict(s=A[6]), dict(gate=None), dict(w=None), dict(w=None, y=None), dict(wp=None),
    dict(w=None, y=None, r2=None, qd=1, q=A[9], qs=A[10]),
    *[{n: ODD} for n in ("x", "res", "wp", "w", "s", "y", "r1", "r2")]], ids=str)
def test_forward_refuses(lib, kw):
    assert fwd(lib, **kw) == INVALID


def test_gate_alignment(lib):
    byte = ctypes.c_void_p(0x10001)
    assert fwd(lib, dict(gate_dtype=16), gate=ODD) == INVALID      # a row gate in fp32
    assert fwd(lib, dict(gate_dtype=0), gate=byte) == INVALID
    for kind in (2, 3):
        assert fwd(lib, dict(gate=kind), gate=ctypes.c_void_p(0x10008)) == INVALID


@pytest.mark.parametrize("kw", [dict(H=12), dict(H=32776), dict(qd=1, q=A[9], qs=A[10], H=64), dict(qd=2, q=A[9], qs=A[10], H=48)], ids=str)
def test_shapes_not_taken(lib, kw):
    assert fwd(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(s=None), dict(r2=None), dict(r1=None), dict(x=None), dict(dx=None), dict(dx=A[10]), dict(T=-1), dict(H=4),
    dict(wt=1), dict(w=None), dict(w=None, dw=None), dict(w=None, dw=None, dy=None, ds=None), dict(wp=None),
    dict(ws=None), dict(n=64), dict(ws=ODD), dict(gate=None), *[{n: ODD} for n in ("dy", "ds", "x", "s", "dx", "dres", "dw", "dwp", "r1", "r2")]],
    ids=str)
def test_backward_refuses(lib, kw):
    assert bwd(lib, **kw) == INVALID


def test_backward_refuses_gradients_of_nothing(lib):
    assert bwd(lib, dict(gate=0), gate=None) == INVALID
    assert bwd(lib, dict(gate=2), dg=ODD) == INVALID and bwd(lib, dict(gate=3), dg=ctypes.c_void_p(0x10008)) == INVALID
    assert bwd(lib, H=20) == UNSUPPORTED and bwd(lib, H=40000) == UNSUPPORTED


def test_no_rows(lib):
    none = dict(x=None, res=None, gate=None, s=None, y=None, r1=None, r2=None, T=0)
    assert fwd(lib, **none) == OK and fwd(lib, H=12, **none) == UNSUPPORTED
    assert fwd(lib, dict(gate=2), **none) == INVALID           # a channel gate is there for no rows too
    assert bwd(lib, dy=None, ds=None, x=None, s=None, gate=None, r1=None, r2=None, dx=None, dres=None, dw=None, dwp=None, dg=None,
               ws=None, n=0, T=0) == OK
    for f in ((0, 128), (-1, 128), (4, 12), (4, 0), (4, 1 << 16)):
        assert lib.moe_sandwich_norm_backward_workspace_bytes(*f) == 0
    assert lib.moe_sandwich_norm_backward_workspace_bytes(4, 128) >= 3 * 4 * 128 * 4


def test_no_config(lib):
    assert fwd(lib, "null") == INVALID and bwd(lib, "null") == INVALID


def test_binding_refuses():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_sandwich_norm(x, x, x[0], 1e-6, x)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_sandwich_norm_backward(x, x, x, x, x[0], x[:, 0], x)
    from combine_moe_dispatch_02_amd import block
    with pytest.raises(ValueError, match="gate_act"):
        block._gate(None, "relu", 0, 2, 128)
    with pytest.raises(ValueError, match="gate has shape"):
        block._gate(torch.zeros(2), "none", 0, 2, 128)
    with pytest.raises(ValueError, match="dtype"):
        block._gate(torch.zeros(2, 1, dtype=torch.float16), "none", 0, 2, 128)


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", [None, "row", "channel", "full"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "tanh"])
def test_oracle_gradients_are_derivatives(post, pre, gate, act):
    """Central differences in float64, without the stream's rounding: error of order h^2 and 1e-16 / h."""
    rng = np.random.default_rng(5)
    T, H, eps = 3, 16, 1e-3
    x, res, d_s, dy = (rng.standard_normal((T, H)) for _ in range(4))
    wp = 1 + 0.2 * rng.standard_normal(H) if post else None
    w = 1 + 0.2 * rng.standard_normal(H) if pre else None
    z = None if gate is None else rng.standard_normal({"row": (T, 1), "channel": (H,), "full": (T, H)}[gate])
    rs, bs = 0.7, 1.3

    def loss(x, res, wp, w, z):
        s, _, _ = ob.sandwich(x, res, wp, z, act, rs, bs, eps)
        y = s * ob.inverse_rms(s, eps) * w if w is not None else 0.0
        return (s * d_s).sum() + (y * dy).sum()

    s, r1, _ = ob.sandwich(x, res, wp, z, act, rs, bs, eps)
    g = ob.sandwich_backward(dy, d_s, x, s, wp, w, z, act, rs, bs, r1, ob.inverse_rms(s, eps))
    if z is not None:
        g["d_gate"] = {"row": g["d_gate"].sum(1, keepdims=True), "channel": g["d_gate"].sum(0), "full": g["d_gate"]}[gate]
    args = [x, res, wp, w, z]
    for at, name in ((0, "dx"), (1, "d_res"), (2, "dwp"), (3, "dw"), (4, "d_gate")):
        if args[at] is None:
            continue
        for i in np.ndindex(args[at].shape):
            d = []
            for h in (1e-5, -1e-5):
                b = [None if v is None else v.copy() for v in args]
                b[at][i] += h
                d.append(loss(*b))
            assert abs((d[0] - d[1]) / 2e-5 - g[name][i]) < 1e-6, (name, i)

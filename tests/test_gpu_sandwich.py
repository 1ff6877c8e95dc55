"""The norms around the residual's addition with gate and scales, and the backward pass, on the GPU.

Forward: both statistics are summed in 64 bits and products and sums are rounded one by one, so with a gate
that is its own factor the stream, rstd, y, codes and scales are compared with the oracle bit for bit. An activation
is off by at most 8 U relative (U = 2^-24; expf and tanhf 2 units in the last place, a sum and a quotient): the stream then is
within 16 U of its terms' magnitudes and a bf16 half step (2^-8), and all that follows is compared bit for bit on the
stream as it was stored.

Backward, against float64 on the same stored inputs. A row's sums add at most 53 terms in a chain (32 values of
a lane, 6 steps in the wave, 15 waves) of at most 8 roundings and an activation: within N = 80 U of the terms' magnitudes. Sums over rows
add at most T + 24 terms. Elementwise chains have at most 12 roundings besides. A slope is f (1 - f) or
1 - f^2 of an f off by 8 U: within 16 U absolutely."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import behind as ob
from oracle import block as obb

from _gpu import say

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
SHAPE = {"row": lambda T, H: (T, 1), "channel": lambda T, H: (H,), "full": lambda T, H: (T, H)}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def same(t, ref):
    return np.array_equal(t.detach().float().cpu().numpy(), np.asarray(ref, dtype=np.float32).reshape(t.shape), equal_nan=True)


def make(T, H, seed, *, post=True, pre=True, gate=None, wdt=BF16, gdt=BF16, res=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=(0.6 * n(T, H)).to(BF16), res=(3 * n(T, H)).to(BF16) if res else None,
             wp=(0.8 + 0.2 * n(H)).to(wdt) if post else None, w=(1 + 0.2 * n(H)).to(wdt) if pre else None,
             gate=None if gate is None else (0.5 + n(*SHAPE[gate](T, H))).to(gdt),
             dy=n(T, H).to(BF16) if pre else None, d_s=n(T, H).to(BF16))
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def forward(d, act="none", rs=1.0, bs=1.0, fmt="bf16", eps=1e-6, peps=1e-5, y=True, stream=None):
    T, H = d["x"].shape
    e = lambda *s, dt=F32: torch.full(s, 7, device="cuda", dtype=dt)  # noqa: E731
    o = dict(s=e(T, H, dt=BF16), y=e(T, H, dt=BF16) if d["w"] is not None and y else None,
             r1=e(T) if d["wp"] is not None else None, r2=e(T) if d["w"] is not None else None, q=None, q_s=None)
    if fmt != "bf16":
        o["q"] = e(T, H, dt=torch.uint8)
        o["q_s"] = moe.quantized_scales(T, H, fmt).fill_(9)
    moe.moe_sandwich_norm(d["x"], d["res"], d["w"], eps, o["s"], o["y"], post_weight=d["wp"], post_eps=peps, gate=d["gate"],
                          gate_act=act, res_scale=rs, branch_scale=bs, post_rstd=o["r1"], rstd=o["r2"], q=o["q"], q_s=o["q_s"],
                          dtype=fmt, stream=stream)
    torch.cuda.synchronize()
    return o


def np32(t):
    return None if t is None else t.detach().float().cpu().numpy()


def check_forward(d, o, act="none", rs=1.0, bs=1.0, fmt="bf16", eps=1e-6, peps=1e-5):
    x, res, wp, gate = (np32(d[k]) for k in ("x", "res", "wp", "gate"))
    if act == "none":
        s, r1 = ob.sandwich_bits(x, res, wp, gate, rs, bs, peps)
        assert same(o["s"], s)
        if wp is not None:
            assert same(o["r1"], r1)
    else:
        ref, r1, p = ob.sandwich(x, res, wp, gate, act, float(np.float32(rs)), float(np.float32(bs)), peps)
        f = ob.gate_act(gate, act) * bs
        terms = np.abs(p * f) + (0 if res is None else np.abs(res.astype(np.float64) * rs))
        assert (np.abs(f64(o["s"]) - ref) <= HALF * np.abs(ref) + 32 * U * terms + 1e-37).all()
    if d["w"] is not None:
        r2, y = ob.sandwich_norm(np32(o["s"]), np32(d["w"]), eps)
        assert same(o["r2"], r2)
        if o["y"] is not None:
            assert same(o["y"], y)
        if fmt != "bf16":
            codes, scales = obb.quantize_rows(y, fmt)
            assert np.array_equal(o["q"].cpu().numpy(), codes)
            assert np.array_equal(o["q_s"].cpu().numpy(), scales)


def backward(d, o, act="none", rs=1.0, bs=1.0, ws=None, stream=None, want=("dx", "d_res", "dw", "dwp", "d_gate")):
    T, H = d["x"].shape
    e = lambda *s, dt=F32: torch.full(s, 7, device="cuda", dtype=dt)  # noqa: E731
    g = dict(dx=e(T, H, dt=BF16), d_res=e(T, H, dt=BF16) if "d_res" in want else None,
             dw=e(H) if d["w"] is not None and "dw" in want else None, dwp=e(H) if d["wp"] is not None and "dwp" in want else None, d_gate=None)
    if d["gate"] is not None and "d_gate" in want:
        g["d_gate"] = e(*d["gate"].shape, dt=F32 if d["gate"].shape == (H,) else d["gate"].dtype)
    if ws is None:
        ws = torch.empty(moe.sandwich_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_sandwich_norm_backward(d["dy"], d["d_s"], d["x"], o["s"], d["w"], o["r2"], g["dx"], g["d_res"], g["dw"], ws,
                                   post_weight=d["wp"], post_rstd=o["r1"], gate=d["gate"], gate_act=act, res_scale=rs, branch_scale=bs,
                                   d_post_weight=g["dwp"], d_gate=g["d_gate"], stream=stream)
    torch.cuda.synchronize()
    return g


def check_backward(d, o, g, act="none", rs=1.0, bs=1.0):
    T, H = d["x"].shape
    rs, bs = float(np.float32(rs)), float(np.float32(bs))
    x, s, dy, d_s, wp, w, z = (f64(t) for t in (d["x"], o["s"], d["dy"], d["d_s"], d["wp"], d["w"], d["gate"]))
    r1 = None if wp is None else f64(o["r1"])[:, None]
    r2 = None if w is None else f64(o["r2"])[:, None]
    ref = ob.sandwich_backward(dy, d_s, x, s, wp, w, z, act, rs, bs, r1, r2)
    N = 80 * U
    mean = lambda v: v.sum(1, keepdims=True) / H  # noqa: E731
    # what the terms of each sum amount to, and how far the sums may be off
    f = np.abs(bs) * (np.ones((1, 1)) if z is None else np.abs(ob.gate_act(z, act)))
    slope = np.zeros((1, 1)) if z is None else np.abs(bs) * np.abs(ob.gate_slope(z, act))
    slope_off = np.abs(bs) * 16 * U
    xh = np.abs(x) if wp is None else np.abs(x * r1)
    p = xh if wp is None else xh * np.abs(wp)
    mag, off = np.abs(d_s) if d_s is not None else np.zeros((T, H)), 0.0
    k_off = 0.0                                         # of sum p f ds over the row, beside what its own terms give
    if w is not None:
        xs, gg = np.abs(s * r2), np.abs(dy * w)
        c2 = mean(gg * xs)
        mag = mag + r2 * (gg + xs * c2)
        off = r2 * xs * N * c2
        k_off = r2 * N * c2 * (p * f * xs).sum(1, keepdims=True)
    ds_off = off + 12 * U * mag
    assert_near(g["d_res"], ref["d_res"], np.abs(rs) * ds_off, HALF)
    dp_off = f * ds_off + 16 * U * f * mag
    k_off = k_off + N * (p * f * mag).sum(1, keepdims=True)
    if wp is not None:
        c1_off = k_off / H
        dx_off = r1 * (np.abs(wp) * dp_off + xh * c1_off + 12 * U * (np.abs(wp) * f * mag + xh * mean(p * f * mag)))
    else:
        dx_off = dp_off
    assert_near(g["dx"], ref["dx"], dx_off, HALF)
    rows = (T + 36) * U
    if g["dw"] is not None:
        assert_near(g["dw"], ref["dw"], rows * np.abs(dy * s * r2).sum(0))
    if g["dwp"] is not None:
        assert_near(g["dwp"], ref["dwp"], (dp_off * xh).sum(0) + rows * (f * mag * xh).sum(0))
    if g["d_gate"] is not None:
        one = np.ones((T, H))
        each = (slope * ds_off + (slope_off + 12 * U * slope) * mag) * p * one
        full = slope * mag * p * one
        half = HALF if g["d_gate"].dtype == BF16 else U
        if z.shape == (T, H):
            assert_near(g["d_gate"], ref["d_gate"], each, half)
        elif z.shape == (H,):
            assert_near(g["d_gate"], ref["d_gate"].sum(0), each.sum(0) + rows * full.sum(0))
        else:
            xs_off = 0.0 if w is None else r2 * N * c2 * (p * xs).sum(1, keepdims=True)
            row = slope * (xs_off + N * (p * mag).sum(1, keepdims=True)) + slope_off * (p * mag).sum(1, keepdims=True)
            assert_near(g["d_gate"], ref["d_gate"].sum(1, keepdims=True), row, half)


def assert_near(t, ref, off, half=0.0):
    got = f64(t)
    ref = np.asarray(ref).reshape(got.shape)
    bad = np.abs(got - ref) > np.broadcast_to(off, got.shape) + half * np.abs(ref) * (1 + HALF) + half * np.broadcast_to(off, got.shape) + 1e-37
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


# every register layout of the kernels: the smallest, odd and largest widths of each
WIDTHS = [8, 24, 128, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("H", WIDTHS)
def test_forward_bits_every_width(H):
    for T, post, gate in ((1, True, "row"), (5, True, "channel"), (6, False, "full"), (3, True, None)):
        say("sandwich", T, H, post, gate)
        d = make(T, H, H + T, post=post, gate=gate, wdt=F32 if H % 16 else BF16, gdt=F32 if T == 6 else BF16)
        check_forward(d, forward(d, rs=0.5, bs=1.5), rs=0.5, bs=1.5)


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
def test_forward_activations(act, gate):
    for T, H in ((1, 8), (7, 520), (33, 4096)):
        for spread in (1.0, 30.0):
            d = make(T, H, T, gate=gate, gdt=F32)
            d["gate"] *= spread                     # far tails of the activation too
            check_forward(d, forward(d, act, 1.0, 0.22), act, 1.0, 0.22)


@pytest.mark.parametrize("fmt,H", [("fp8", 128), ("fp8", 1152), ("fp8", 4096), ("fp8", 16384), ("mxfp4", 32), ("mxfp4", 544),
                                   ("mxfp4", 4128), ("mxfp4", 7168), ("mxfp4", 32768)])
def test_codes(fmt, H):
    for T, gate, y in ((1, "row", True), (9, "channel", False), (4, None, True)):
        d = make(T, H, T + 3, gate=gate)
        check_forward(d, forward(d, fmt=fmt, y=y), fmt=fmt)


def test_forward_without_parts():
    for post in (True, False):
        for pre in (True, False):
            for res in (True, False):
                d = make(5, 520, 2, post=post, pre=pre, res=res, gate="row")
                check_forward(d, forward(d, rs=3.0), rs=3.0)


def test_values_that_are_not_finite():
    d = make(6, 264, 3, gate="full")
    d["x"][0, 3], d["x"][1, 5], d["res"][2, 7], d["gate"][3, 9] = float("inf"), float("nan"), float("-inf"), float("nan")
    d["x"][4] = 0
    d["gate"][5, 11] = float("inf")
    o = forward(d)
    check_forward(d, o)
    assert torch.isfinite(o["s"][4].float()).all() and torch.isnan(o["s"][:2].float()).any(1).all()


@pytest.mark.parametrize("H", WIDTHS)
def test_backward_every_width(H):
    for T, post, pre, gate in ((1, True, True, "row"), (5, True, True, "channel"), (6, False, True, "full"), (3, True, False, None)):
        say("sandwich backward", T, H, post, pre, gate)
        d = make(T, H, H + T, post=post, pre=pre, gate=gate, wdt=F32 if H % 16 else BF16)
        o = forward(d, rs=0.5, bs=1.5)
        check_backward(d, o, backward(d, o, rs=0.5, bs=1.5), rs=0.5, bs=1.5)


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", [None, "row", "channel", "full"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "tanh"])
def test_backward_every_kind(post, pre, gate, act):
    for T, H, gdt in ((37, 520, BF16), (130, 1032, F32), (11, 264, F32)):
        d = make(T, H, T, post=post, pre=pre, gate=gate, gdt=gdt)
        o = forward(d, act, 0.7, 1.3)
        check_backward(d, o, backward(d, o, act, 0.7, 1.3), act, 0.7, 1.3)


@pytest.mark.parametrize("T,H", [(4500, 264), (1100, 2048), (1030, 4096), (700, 8192)])
def test_backward_several_rows_a_workgroup(T, H):
    d = make(T, H, 1, gate="channel")
    o = forward(d, "sigmoid")
    check_backward(d, o, backward(d, o, "sigmoid"), "sigmoid")


def test_backward_without_the_streams_gradient_and_of_parts():
    d = make(9, 520, 4, gate="row")
    d["d_s"] = None
    o = forward(d)
    whole = backward(d, o)
    check_backward(d, o, whole)
    some = backward(d, o, want=())
    assert torch.equal(some["dx"], whole["dx"])


def test_in_place_and_rows_behind():
    T, H = 5, 4104
    for wide in (H, 16392):                       # rows held in registers, and read twice
        d = make(T, wide, 8, gate="full")
        o = forward(d)
        g = backward(d, o)
        big = {k: torch.cat([d[k], torch.full_like(d[k][:1], 3)]) for k in ("x", "res", "dy", "d_s")}
        x, res = big["x"][:T], big["res"][:T]
        moe.moe_sandwich_norm(x, res, d["w"], 1e-6, res, x, post_weight=d["wp"], post_eps=1e-5, gate=d["gate"])
        assert torch.equal(res, o["s"]) and torch.equal(x, o["y"])
        x.copy_(d["x"])
        dg = d["gate"].clone()
        ws = torch.empty(moe.sandwich_norm_backward_workspace_bytes(T, wide), dtype=torch.uint8, device="cuda")
        dw, dwp = torch.empty(wide, device="cuda"), torch.empty(wide, device="cuda")
        moe.moe_sandwich_norm_backward(big["dy"][:T], big["d_s"][:T], x, o["s"], d["w"], o["r2"], big["dy"][:T], big["d_s"][:T], dw, ws,
                                       post_weight=d["wp"], post_rstd=o["r1"], gate=dg, d_post_weight=dwp, d_gate=dg)
        assert torch.equal(big["dy"][:T], g["dx"]) and torch.equal(big["d_s"][:T], g["d_res"]) and torch.equal(dg, g["d_gate"])
        assert torch.equal(dw, g["dw"]) and torch.equal(dwp, g["dwp"])
        assert all((v[T] == 3).all() for v in big.values())


def test_no_rows():
    d = make(0, 264, 1, gate="channel")
    o = forward(d)
    g = backward(d, o)
    assert (g["dw"] == 0).all() and (g["dwp"] == 0).all() and (g["d_gate"] == 0).all()


def test_same_bits_again_and_on_another_stream():
    d = make(300, 4096, 5, gate="channel")
    o = forward(d, "sigmoid")
    g = backward(d, o, "sigmoid")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o2 = forward(d, "sigmoid", stream=st)
    st.synchronize()
    g2 = backward(d, o2, "sigmoid", stream=st)
    for a, b in ((o, o2), (g, g2)):
        assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


def test_graph_replays():
    d = make(70, 1032, 6, gate="row")
    o = forward(d, "tanh")
    ref_o, ref_g = {k: v.clone() for k, v in o.items() if v is not None}, backward(d, o, "tanh")
    ws = torch.empty(moe.sandwich_norm_backward_workspace_bytes(70, 1032), dtype=torch.uint8, device="cuda")
    g = {k: torch.zeros_like(v) for k, v in ref_g.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_sandwich_norm(d["x"], d["res"], d["w"], 1e-6, o["s"], o["y"], post_weight=d["wp"], post_eps=1e-5, gate=d["gate"],
                              gate_act="tanh", post_rstd=o["r1"], rstd=o["r2"])
        moe.moe_sandwich_norm_backward(d["dy"], d["d_s"], d["x"], o["s"], d["w"], o["r2"], g["dx"], g["d_res"], g["dw"], ws,
                                       post_weight=d["wp"], post_rstd=o["r1"], gate=d["gate"], gate_act="tanh",
                                       d_post_weight=g["dwp"], d_gate=g["d_gate"])
    for _ in range(4):
        for v in list(g.values()) + [o["s"], o["y"], o["r1"], o["r2"]]:
            v.fill_(5)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g[k], ref_g[k]) for k in g) and all(torch.equal(o[k], ref_o[k]) for k in ref_o)


def test_past_the_grid_and_past_4_gib():
    """More rows than workgroups, and arrays over 2^32 bytes: rows alone give the bits they give among all."""
    for T, H in ((300000, 8), (70000, 32768)):
        say("sandwich", T, H)
        g = torch.Generator(device="cuda").manual_seed(2)
        d = dict(x=torch.randn(T, H, generator=g, device="cuda", dtype=BF16), res=torch.randn(T, H, generator=g, device="cuda", dtype=BF16),
                 wp=torch.ones(H, device="cuda", dtype=BF16), w=torch.ones(H, device="cuda", dtype=BF16),
                 gate=torch.randn(T, 1, generator=g, device="cuda"))
        d["dy"], d["d_s"] = d["res"], d["x"]
        o = forward(d, "sigmoid")
        gr = backward(d, o, "sigmoid", want=("d_res", "d_gate"))
        at = torch.tensor([0, 65535, 65536, T - 2, T - 1], device="cuda")
        few = {k: v[at].contiguous() if v.shape[0] == T else v for k, v in d.items()}
        oo = forward(few, "sigmoid")
        gg = backward(few, oo, "sigmoid", want=("d_res", "d_gate"))
        assert all(torch.equal(o[k][at], oo[k]) for k in ("s", "y", "r1", "r2"))
        assert all(torch.equal(gr[k][at], gg[k]) for k in ("dx", "d_res", "d_gate"))
        del d, o, gr

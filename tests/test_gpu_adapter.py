"""Low-rank adapters of many requests and their gradients on the GPU, against float64.

Tolerances (U = 2^-24): a sum of K exact products in fp32, in any order, is off by at most K U of the sum of their
magnitudes; sums with random signs by about U sqrt(K / 2) of the result's norm, of which four times
are taken as a second, tighter bound on the whole array. v enters the second product as two bf16 numbers, off
by 2^-18 of its magnitude, whose 2 R products add 2 R U; out and dx end in a bf16 half step (2^-8). dA and dB take three bf16
numbers (all bits): 3 sums' additions a row, U each; with partial sums of chunks not more."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from oracle import behind as ob

from _gpu import say

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(T, n, K, N, R, seed=0, ids="mixed", ranks=False, scale=True):
    g = torch.Generator().manual_seed(seed * 1000 + T + K)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    i = torch.randint(-1, n, (T,), generator=g)
    if ids == "runs":
        i = i.sort()[0].roll(T // 3)
    elif isinstance(ids, list):
        i = torch.tensor(ids)
    d = dict(x=r(T, K).to(BF16), a=(r(n, R, K) / K ** 0.5).to(BF16), b=(r(n, N, R) / R ** 0.5).to(BF16), ids=i.to(torch.int32),
             scale=0.5 + torch.rand(n, generator=g) if scale else None, ranks=None, base=r(T, N).to(BF16), dout=r(T, N).to(BF16),
             dx_base=r(T, K).to(BF16))
    if ranks:
        k = torch.randint(0, R + 1, (n,), generator=g)
        d["ranks"] = k.to(torch.int32)
        for e in range(n):                       # what is past an adapter's rank is not looked at
            d["a"][e, k[e]:] = NAN
            d["b"][e, :, k[e]:] = NAN
    d["x"][i < 0] = NAN                          # nor are rows without an adapter
    d["dout"][i < 0] = NAN
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def make_plan(d, tile, begin=0):
    T, n = d["x"].shape[0], d["a"].shape[0]
    plan, ws = moe.Plan.allocate(T, 1, begin, n, tile), moe.Workspace(T, 1, n, tile)
    moe.moe_plan((d["ids"] + begin).view(T, 1), plan, ws)
    return plan


def forward(d, plan=None, base="base", v=True, stream=None, **kw):
    T, K = d["x"].shape
    R, N = d["a"].shape[1], d["b"].shape[1]
    o = dict(out=torch.full((T, N), 7, dtype=BF16, device="cuda"), v=torch.full((T, R), 7.0, device="cuda") if v else None)
    ws = torch.full((moe.adapter_workspace_bytes(T, K, R),), 255, dtype=torch.uint8, device="cuda")
    by = {"plan": plan} if plan is not None else {"ids": d["ids"]}
    moe.moe_adapter(d["x"], d["a"], d["b"], o["out"], ws, base=d[base] if base else None, scale=d["scale"], ranks=d["ranks"], v=o["v"],
                    stream=stream, **by, **kw)
    torch.cuda.synchronize()
    return o


def magnitudes(d, ids):
    """Per row: |A| |x| (sums of magnitudes behind v), with nothing where there is no adapter."""
    a, x = np.nan_to_num(np.abs(f64(d["a"]))), np.nan_to_num(np.abs(f64(d["x"])))
    m = np.zeros((x.shape[0], a.shape[1]))
    for e in range(a.shape[0]):
        t = np.nonzero(ids == e)[0]
        m[t] = x[t] @ a[e].T
    return m


def per_row(m, table, ids, transposed=False):
    """table[e] (or its transpose) times m[t], row by row, magnitudes."""
    w = np.nan_to_num(np.abs(f64(table)))
    out = np.zeros((m.shape[0], w.shape[2] if transposed else w.shape[1]))
    for e in range(w.shape[0]):
        t = np.nonzero(ids == e)[0]
        out[t] = m[t] @ (w[e] if transposed else w[e].T)
    return out


def near(t, ref, off, half=0.0):
    got = f64(t)
    bad = ~(np.abs(got - ref) <= off * (1 + half) + half * np.abs(ref) * (1 + HALF))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def tight(t, ref, K):
    """The whole array's error against four times what random signs give (and 2^-17 of a split below it)."""
    if ref.size >= 64 and np.abs(ref).max() > 0:
        assert np.linalg.norm(f64(t) - ref) <= (4 * U * K ** 0.5 + 16 * U) * np.linalg.norm(ref)


def check_forward(d, o, base="base"):
    ids = d["ids"].cpu().numpy()
    K, R = d["x"].shape[1], d["a"].shape[1]
    clean = lambda t: np.nan_to_num(f64(t))  # noqa: E731
    scale = f64(d["scale"])
    ranks = None if d["ranks"] is None else d["ranks"].cpu().numpy()
    ref, v = ob.adapter(clean(d["x"]), ids, clean(d["a"]), clean(d["b"]), scale, ranks, f64(d[base]) if base else None)
    on = ids >= 0
    m = magnitudes(d, ids)
    if o["v"] is not None:
        near(o["v"][torch.from_numpy(on).cuda()], v[on], K * U * m[on])
        tight(o["v"][torch.from_numpy(on).cuda()], v[on], K)
    s = np.ones(len(ids)) if scale is None else np.where(on, np.abs(scale[np.where(on, ids, 0)]), 0.0)
    delta = s[:, None] * per_row(K * U * m + (2.0 ** -18 + (2 * R + 4) * U) * np.abs(v), d["b"], ids)
    near(o["out"], ref, delta + 4 * U * np.abs(ref), HALF)
    if (~on).any():
        rows = torch.from_numpy(~on).cuda()
        assert torch.equal(o["out"][rows], d[base][rows] if base else torch.zeros_like(o["out"][rows]))
    return v


SIZES = [(1, 1, 8, 8, 8), (1, 4, 64, 72, 16), (5, 3, 40, 24, 24), (64, 64, 256, 136, 64), (33, 2, 520, 264, 40), (64, 1, 4096, 512, 128),
         (17, 5, 72, 1032, 256), (50, 7, 1032, 40, 136), (64, 1000, 128, 128, 8), (31, 3, 2056, 2056, 72)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("ranks", [False, True])
def test_forward_by_ids(size, ranks):
    say("adapter ids", size, ranks)
    d = make(*size, ranks=ranks, scale=ranks)
    check_forward(d, forward(d))
    check_forward(d, forward(d, base=None, v=False), None)


@pytest.mark.parametrize("size", SIZES + [(300, 5, 264, 136, 24), (1021, 32, 512, 200, 64), (4100, 3, 72, 72, 16), (700, 1, 136, 2056, 136)], ids=str)
@pytest.mark.parametrize("tile", [16, 32, 128])
def test_forward_by_plan(size, tile):
    say("adapter plan", size, tile)
    for ids in ("mixed", "runs"):
        d = make(*size, ids=ids, ranks=ids == "runs")
        o = forward(d, make_plan(d, tile))
        check_forward(d, o)
        if size[0] <= 64:                        # a row's sums are the same however rows are grouped
            p = forward(d)
            on = d["ids"] >= 0
            assert torch.equal(o["out"], p["out"]) and torch.equal(o["v"][on], p["v"][on])


def test_all_rows_one_adapter_and_none():
    for ids in ([0] * 64, [-1] * 64, [2] * 33 + [-5] * 30 + [99]):
        d = make(64, 3, 128, 64, 32, ids=ids)
        if 99 in ids:
            d["x"][63] = NAN
        check = dict(d)
        check["ids"] = torch.where((d["ids"] >= 0) & (d["ids"] < 3), d["ids"], -1)
        check_forward(check, forward(d))
        check_forward(check, forward(d, make_plan(d, 64)))


def test_begin():
    d = make(40, 4, 64, 64, 16)
    ref = forward(d)
    far = dict(d, ids=d["ids"] + 100)
    got = forward(far, id_begin=100)
    plan = forward(d, make_plan(d, 16, begin=100))
    on = d["ids"] >= 0
    for o in (got, plan):
        assert torch.equal(o["out"], ref["out"]) and torch.equal(o["v"][on], ref["v"][on])


def test_columns_of_wider_arrays_in_place_and_rows_behind():
    for T, n, K, N, R, tile in ((40, 4, 72, 136, 24, None), (600, 3, 520, 648, 40, 32)):
        d = make(T, n, K, N, R, ranks=True)
        plan = make_plan(d, tile) if tile else None
        ref = forward(d, plan)
        wide = {k: torch.full((T + 1, w + 64), 3, dtype=BF16, device="cuda") for k, w in (("x", K), ("base", N), ("out", N))}
        col = lambda k, w: wide[k][:T, 16:16 + w]  # noqa: E731
        col("x", K).copy_(d["x"])
        col("base", N).copy_(d["base"])
        ws = torch.empty(moe.adapter_workspace_bytes(T, K, R), dtype=torch.uint8, device="cuda")
        by = {"plan": plan} if plan is not None else {"ids": d["ids"]}
        more = dict(scale=d["scale"], ranks=d["ranks"], **by)
        moe.moe_adapter(col("x", K), d["a"], d["b"], col("out", N), ws, base=col("base", N), **more)
        moe.moe_adapter(col("x", K), d["a"], d["b"], col("base", N), ws, base=col("base", N), **more)
        torch.cuda.synchronize()
        for k in ("out", "base"):
            assert torch.equal(col(k, N), ref["out"])
            assert (wide[k][:, :16] == 3).all() and (wide[k][:, 16 + N:] == 3).all() and (wide[k][T] == 3).all()
        if plan is None:
            continue
        # the gradients' arrays too
        g = backward(d, ref, plan)
        dwide = {k: torch.full((T + 1, w + 64), 3, dtype=BF16, device="cuda") for k, w in (("dout", N), ("dx", K))}
        dwide["dout"][:T, 8:8 + N] = d["dout"]
        dwide["dx"][:T, 24:24 + K] = d["dx_base"]
        dx = dwide["dx"][:T, 24:24 + K]
        bws = torch.empty(moe.adapter_backward_workspace_bytes(T, n, K, N, R), dtype=torch.uint8, device="cuda")
        da, db = torch.empty_like(g["da"]), torch.empty_like(g["db"])
        moe.moe_adapter_backward(dwide["dout"][:T, 8:8 + N], col("x", K), ref["v"], d["a"], d["b"], plan, bws, da, db, dx, dx_base=dx,
                                 scale=d["scale"], ranks=d["ranks"])
        torch.cuda.synchronize()
        assert torch.equal(dx, g["dx"]) and torch.equal(da, g["da"]) and torch.equal(db, g["db"])
        assert (dwide["dx"][:, :24] == 3).all() and (dwide["dx"][:, 24 + K:] == 3).all() and (dwide["dx"][T] == 3).all()


def backward(d, o, plan, want=("dx", "da", "db"), base=True, ws=None, stream=None):
    T, K = d["x"].shape
    (n, R), N = d["a"].shape[:2], d["b"].shape[1]
    e = lambda *s, dt=F32: torch.full(s, 7, device="cuda", dtype=dt)  # noqa: E731
    g = dict(dx=e(T, K, dt=BF16) if "dx" in want else None, da=e(n, R, K) if "da" in want else None, db=e(n, N, R) if "db" in want else None)
    if ws is None:
        ws = torch.full((moe.adapter_backward_workspace_bytes(T, n, K, N, R),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_adapter_backward(d["dout"], d["x"], o["v"], d["a"], d["b"], plan, ws, g["da"], g["db"], g["dx"],
                             dx_base=d["dx_base"] if base and "dx" in want else None, scale=d["scale"], ranks=d["ranks"], stream=stream)
    torch.cuda.synchronize()
    return g


def check_backward(d, o, g, base=True):
    ids = d["ids"].cpu().numpy()
    on = ids >= 0
    T, K = d["x"].shape
    (n, R), N = d["a"].shape[:2], d["b"].shape[1]
    clean = lambda t: np.nan_to_num(f64(t))  # noqa: E731
    scale = np.ones(n) if d["scale"] is None else f64(d["scale"])
    ranks = None if d["ranks"] is None else d["ranks"].cpu().numpy()
    x, dout, v = clean(d["x"]), clean(d["dout"]), np.where(on[:, None], f64(o["v"]), 0.0)
    dx, da, db = ob.adapter_backward(dout, x, v, ids, clean(d["a"]), clean(d["b"]), scale, ranks, f64(d["dx_base"]) if base else None)
    s = np.where(on, np.abs(scale[np.where(on, ids, 0)]), 0.0)[:, None]
    dv_mag = s * per_row(np.abs(dout), d["b"], ids, transposed=True)
    dv_off = (N + 2) * U * dv_mag
    off = per_row(dv_off + (2.0 ** -18 + (2 * R + 4) * U) * dv_mag, d["a"], ids, transposed=True)
    if g["dx"] is not None:
        near(g["dx"], dx, off + 4 * U * np.abs(dx), HALF)
        if (~on).any():
            rows = torch.from_numpy(~on).cuda()
            assert torch.equal(g["dx"][rows], d["dx_base"][rows] if base else torch.zeros_like(g["dx"][rows]))
    da_off, db_off = np.zeros(da.shape), np.zeros(db.shape)
    for e in range(n):
        t = np.nonzero(ids == e)[0]
        k = (3 * len(t) + 16) * U
        da_off[e] = (dv_off[t] + k * dv_mag[t]).T @ np.abs(x[t])
        db_off[e] = scale[e] * k * (np.abs(dout[t]).T @ np.abs(v[t]))
    if g["da"] is not None:
        near(g["da"], da, da_off)
        tight(g["da"], da, N + 3 * T)
    if g["db"] is not None:
        near(g["db"], db, db_off)
        tight(g["db"], db, 3 * T)


@pytest.mark.parametrize("size", [(1, 1, 8, 8, 8), (5, 3, 40, 24, 24), (64, 64, 256, 136, 64), (33, 2, 520, 264, 40), (300, 5, 264, 136, 24),
                                  (17, 5, 72, 1032, 256), (1021, 32, 512, 200, 64), (2600, 3, 72, 136, 16), (700, 1, 136, 2056, 136),
                                  (64, 1000, 128, 128, 8), (3000, 2, 264, 72, 64)], ids=str)
@pytest.mark.parametrize("tile", [16, 32, 128])
def test_backward(size, tile):
    say("adapter backward", size, tile)
    for ids in ("mixed", "runs"):
        d = make(*size, ids=ids, ranks=ids == "runs", scale=tile != 16)
        plan = make_plan(d, tile)
        o = forward(d, plan)
        check_backward(d, o, backward(d, o, plan))
        check_backward(d, o, backward(d, o, plan, base=False), base=False)


def test_backward_of_parts_and_without_adapters():
    d = make(300, 4, 136, 72, 24)
    plan = make_plan(d, 32)
    o = forward(d, plan)
    whole = backward(d, o, plan)
    for want in (("dx",), ("da",), ("db",), ("dx", "db")):
        g = backward(d, o, plan, want)
        assert all(torch.equal(g[k], whole[k]) for k in want)
    d = make(80, 4, 136, 72, 24, ids=[-1] * 80)
    plan = make_plan(d, 32)
    g = backward(d, forward(d, plan), plan)
    assert (g["da"] == 0).all() and (g["db"] == 0).all() and torch.equal(g["dx"], d["dx_base"])


def test_no_rows():
    d = make(0, 3, 64, 48, 16)
    forward(d)
    da, db = torch.full((3, 16, 64), 7.0, device="cuda"), torch.full((3, 48, 16), 7.0, device="cuda")
    moe.moe_adapter_backward(d["dout"], None, None, d["a"], d["b"], None, None, da, db)
    torch.cuda.synchronize()
    assert (da == 0).all() and (db == 0).all()


def test_infinite_values_stay_in_their_rows():
    d = make(60, 3, 128, 64, 16, ids=[0, 1, 2] * 20)
    d["x"][7, 3] = float("inf")
    d["x"][8, 5] = NAN
    ok = torch.ones(60, dtype=torch.bool)
    ok[7] = ok[8] = False
    ref = forward(dict(d, x=torch.where(torch.isfinite(d["x"]), d["x"], 0)))
    o = forward(d)
    assert torch.equal(o["out"][ok.cuda()], ref["out"][ok.cuda()]) and not torch.isfinite(o["out"][7:9].float()).any()


def test_same_bits_again_and_on_another_stream():
    d = make(2100, 5, 520, 264, 40, ids="runs")
    plan = make_plan(d, 32)
    torch.cuda.synchronize()
    o = forward(d, plan)
    g = backward(d, o, plan)
    st = torch.cuda.Stream()
    o2 = forward(d, plan, stream=st)
    g2 = backward(d, o2, plan, stream=st)
    on = d["ids"] >= 0
    assert torch.equal(o["out"], o2["out"]) and torch.equal(o["v"][on], o2["v"][on])
    assert all(torch.equal(g[k], g2[k]) for k in g)


def test_graph_replays():
    """Plan, forward and backward captured; rows change their adapters between replays."""
    T, n, K, N, R = 300, 4, 264, 136, 24
    d = make(T, n, K, N, R)
    d["x"], d["dout"] = torch.nan_to_num(d["x"]), torch.nan_to_num(d["dout"])
    plan, pws = moe.Plan.allocate(T, 1, 0, n, 16), moe.Workspace(T, 1, n, 16)
    ids = d["ids"].clone()
    out, v = torch.empty(T, N, dtype=BF16, device="cuda"), torch.zeros(T, R, device="cuda")
    dx, da, db = torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(n, R, K, device="cuda"), torch.empty(n, N, R, device="cuda")
    ws = torch.empty(moe.adapter_workspace_bytes(T, K, R), dtype=torch.uint8, device="cuda")
    bws = torch.empty(moe.adapter_backward_workspace_bytes(T, n, K, N, R), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_plan(ids.view(T, 1), plan, pws)
        moe.moe_adapter(d["x"], d["a"], d["b"], out, ws, base=d["base"], plan=plan, scale=d["scale"], v=v)
        moe.moe_adapter_backward(d["dout"], d["x"], v, d["a"], d["b"], plan, bws, da, db, dx, dx_base=d["dx_base"], scale=d["scale"])
    for i in range(4):
        ids.copy_(d["ids"].roll(7 * i))
        ws.fill_(255)
        bws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        now = dict(d, ids=ids)
        eager = make_plan(now, 16)
        o = forward(now, eager)
        g = backward(now, o, eager)
        assert torch.equal(out, o["out"]) and torch.equal(dx, g["dx"]) and torch.equal(da, g["da"]) and torch.equal(db, g["db"])


def test_token_graph_by_ids():
    d = make(9, 5, 512, 264, 16)
    d["x"] = torch.nan_to_num(d["x"])
    ids, out = d["ids"].clone(), torch.empty(9, 264, dtype=BF16, device="cuda")
    ws = torch.empty(moe.adapter_workspace_bytes(9, 512, 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapter(d["x"], d["a"], d["b"], out, ws, base=d["base"], ids=ids, scale=d["scale"])
    for i in range(4):
        ids.copy_(d["ids"].roll(i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, forward(dict(d, ids=ids))["out"])


def test_past_4_gib():
    """Row offsets over 2^32 bytes in x, out, dout and dx."""
    T, K, N, R, n = 70000, 32768, 32768, 8, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    d = dict(x=r(T, K), a=r(n, R, K) / 128, b=r(n, N, R), scale=None, ranks=None, base=None, ids=(torch.arange(T, device="cuda") % n).to(torch.int32))
    d["dout"] = d["x"]
    plan = make_plan(d, 128)
    say("adapter past 4 GiB")
    o = forward(d, plan, base=None)
    gr = backward(d, o, plan, want=("dx",), base=False)
    at = torch.tensor([0, 1, 65535, 65536, T - 2, T - 1], device="cuda")
    few = dict(d, x=d["x"][at].contiguous(), dout=d["dout"][at].contiguous(), ids=d["ids"][at].contiguous())
    host = {k: f64(v) if v is not None and k != "ids" else v for k, v in few.items()}
    ids = few["ids"].cpu().numpy()
    ref, v = ob.adapter(host["x"], ids, host["a"], host["b"])
    few_o = dict(out=o["out"][at], v=o["v"][at])
    del o, d
    check_forward(few, few_o, None)
    few["dx_base"] = None
    check_backward(few, few_o, dict(dx=gr["dx"][at], da=None, db=None), base=False)

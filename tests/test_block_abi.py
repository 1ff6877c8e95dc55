"""The operators around the layer (include/moe355_block.h) export what the header declares and
refuse bad arguments before anything is enqueued -- all without a GPU (no call here reaches a
launch), and their Python binding refuses what the C ABI cannot see (shapes, types, devices)."""
import ctypes
import os
import re

import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import oracle
from combine_moe_dispatch_02_amd import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = _abi.MOE_OK, _abi.MOE_ERR_INVALID, _abi.MOE_ERR_UNSUPPORTED
A = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]     # never dereferenced
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        pytest.fail("libmoe355.so is not built (run __graft_entry__.build())")
    return _abi.load()


def test_header_and_signatures_agree(lib):
    text = open(os.path.join(ROOT, "include", "moe355_block.h")).read()
    names = set(re.findall(r"MOE355_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text))
    assert names == {n for n, _, _ in _abi.BLOCK_SIGNATURES}
    assert not names & {n for n, _, _ in _abi.SIGNATURES}
    for n in names:
        assert hasattr(lib, n)


def norm(lib, x=A[0], res=A[1], w=A[2], wt=_abi.MOE_BF16, T=4, H=128, eps=1e-6, s=A[3], y=A[4], rstd=A[5], qd=0, q=None,
         qs=None):
    return lib.moe_rmsnorm(x, res, w, wt, T, H, eps, s, y, rstd, qd, q, qs, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(y=None), dict(T=-1), dict(H=0), dict(H=7), dict(wt=7), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(qd=9), dict(q=A[6]), dict(qs=A[6]), dict(qd=1, q=A[6]),
    dict(qd=2, qs=A[6]), dict(res=None), dict(s=A[4]), dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(s=ODD), dict(y=ODD),
    dict(rstd=ODD), dict(qd=1, q=ODD, qs=A[7]), dict(qd=1, q=A[6], qs=ODD)], ids=str)
def test_norm_refuses(lib, kw):
    assert norm(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(H=12), dict(H=32776), dict(qd=1, q=A[6], qs=A[7], H=64),
                                dict(qd=2, q=A[6], qs=A[7], H=48)], ids=str)
def test_norm_shapes_it_does_not_take(lib, kw):
    assert norm(lib, **kw) == UNSUPPORTED


def test_norm_of_no_rows(lib):
    assert norm(lib, x=None, res=None, s=None, y=None, rstd=None, T=0) == OK
    assert norm(lib, x=None, res=None, s=None, y=None, rstd=None, T=0, H=12) == UNSUPPORTED
    assert lib.moe_rmsnorm_backward(None, None, A[2], 0, None, None, 0, 128, None, None, None, 0, None) == OK
    for f in ((0, 128), (-1, 128), (4, 12), (4, 0), (4, 1 << 16)):
        assert lib.moe_rmsnorm_backward_workspace_bytes(*f) == 0
    assert lib.moe_rmsnorm_backward_workspace_bytes(4, 128) >= 4 * 128 * 4


@pytest.mark.parametrize("kw,rc", [
    (dict(dy=None), INVALID), (dict(s=None), INVALID), (dict(w=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None), INVALID), (dict(ws=None), INVALID), (dict(n=0), INVALID), (dict(T=-3), INVALID), (dict(wt=2), INVALID),
    (dict(dy=ODD), INVALID), (dict(dx=ODD), INVALID), (dict(dr=ODD), INVALID), (dict(ws=ODD), INVALID),
    (dict(H=20), UNSUPPORTED), (dict(H=40000), UNSUPPORTED)], ids=str)
def test_norm_backward_refuses(lib, kw, rc):
    a = dict(dy=A[0], s=A[1], w=A[2], wt=0, rstd=A[3], dr=A[4], T=4, H=128, dx=A[5], dw=A[6], ws=A[7], n=BIG)
    a.update(kw)
    assert lib.moe_rmsnorm_backward(a["dy"], a["s"], a["w"], a["wt"], a["rstd"], a["dr"], a["T"], a["H"], a["dx"], a["dw"],
                                    a["ws"], a["n"], None) == rc


ROUTER_BAD = [
    (dict(E=0), {}), (dict(E=1025), {}), (dict(K=0), {}), (dict(K=17), {}), (dict(K=9), {}), (dict(T=-1), {}),
    (dict(lt=5), {}), (dict(logits=None), {}), (dict(idx=None), {}), (dict(wt=None), {}), (dict(logits=ODD), {}),
    (dict(idx=ODD), {}), (dict(wt=ODD), {}), (dict(lt=0, logits=ctypes.c_void_p(0x10008)), {}),
    ({}, dict(score=2)), ({}, dict(normalize=2)), ({}, dict(groups=0)), ({}, dict(groups=3)), (dict(E=130), dict(groups=65)),
    ({}, dict(topk_groups=0)), ({}, dict(topk_groups=2)), ({}, dict(group_top=0)), ({}, dict(group_top=3)),
    ({}, dict(scale=float("inf"))), ({}, dict(scale=float("nan"))), (dict(K=3), dict(groups=4, topk_groups=1))]


@pytest.mark.parametrize("kw,cfg", ROUTER_BAD, ids=str)
def test_router_refuses(lib, kw, cfg):
    c = dict(score=0, normalize=1, groups=1, topk_groups=1, group_top=1, scale=1.0)
    c.update(cfg)
    c = _abi.RouterConfigT(*c.values())
    a = dict(logits=A[0], lt=_abi.MOE_F32, T=4, E=8, K=2, idx=A[1], wt=A[2])
    a.update(kw)
    assert lib.moe_router_topk(a["logits"], a["lt"], None, a["T"], a["E"], a["K"], ctypes.byref(c), a["idx"], a["wt"],
                               None) == INVALID
    assert lib.moe_router_topk_backward(a["wt"], a["logits"], a["lt"], a["idx"], a["T"], a["E"], a["K"], ctypes.byref(c),
                                        A[5], None) == INVALID


def test_router_of_no_rows_and_without_config(lib):
    c = _abi.RouterConfigT(0, 1, 1, 1, 1, 1.0)
    assert lib.moe_router_topk(None, _abi.MOE_F32, None, 0, 8, 2, ctypes.byref(c), None, None, None) == OK
    assert lib.moe_router_topk_backward(None, None, _abi.MOE_F32, None, 0, 8, 2, ctypes.byref(c), None, None) == OK
    assert lib.moe_router_topk(A[0], _abi.MOE_F32, None, 4, 8, 2, None, A[1], A[2], None) == INVALID
    assert lib.moe_router_topk(A[0], _abi.MOE_F32, ODD, 4, 8, 2, ctypes.byref(c), A[1], A[2], None) == INVALID
    assert lib.moe_router_topk_backward(A[0], A[1], _abi.MOE_F32, A[2], 4, 8, 2, ctypes.byref(c), None, None) == INVALID


def _plan(**kw):
    f = dict(T=64, K=2, expert_begin=0, E_local=8, tile=16, rows_cap=oracle.pool_rows_bound(64, 2, 8, 16))
    f.update(kw)
    return _abi.PlanT(f["T"], f["K"], f["expert_begin"], f["E_local"], f["tile"], f["rows_cap"],
                      0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), INVALID), (dict(qs=None), INVALID), (dict(pool=None), INVALID), (dict(ps=None), INVALID),
    (dict(ws=None), INVALID), (dict(dt=0), INVALID), (dict(dt=5), INVALID), (dict(epoch=0), INVALID), (dict(rows=200), INVALID),
    (dict(rows=-16), INVALID), (dict(q=ODD), INVALID), (dict(pool=ODD), INVALID), (dict(qs=ODD), INVALID), (dict(n=64), INVALID),
    (dict(H=4), INVALID), (dict(H=192), UNSUPPORTED), (dict(dt=2, H=48), UNSUPPORTED), (dict(plan=dict(T=0)), INVALID),
    (dict(plan=dict(tile=24)), INVALID)], ids=str)
def test_dispatch_quantized_refuses(lib, kw, rc):
    a = dict(q=A[0], qs=A[1], H=128, dt=1, rows=240, pool=A[2], ps=A[3], epoch=1, ws=A[4], n=BIG, plan={})
    a.update(kw)
    p = _plan(**a["plan"])
    assert lib.moe_dispatch_quantized(a["q"], a["qs"], a["H"], a["dt"], ctypes.byref(p), a["rows"], a["pool"], a["ps"],
                                      a["epoch"], a["ws"], a["n"], None) == rc


DECODE = dict(x=A[0], xs=A[1], dt=2, T=4, H=256, I=128, K=2, begin=0, E=8, idx=A[2], wt=A[3], w1=A[4], w1s=A[5], w2=A[6],
              w2s=A[7], ws=A[8], n=BIG, out=A[9])


def decode(lib, **kw):
    a = dict(DECODE, **kw)
    return lib.moe_expert_ffn_decode(a["x"], a["xs"], a["dt"], a["T"], a["H"], a["I"], a["K"], a["begin"], a["E"], a["idx"],
                                     a["wt"], a["w1"], a["w1s"], a["w2"], a["w2s"], a["ws"], a["n"], a["out"], None)


@pytest.mark.parametrize("kw,rc", [
    *[({n: None}, INVALID) for n in ("x", "xs", "idx", "wt", "w1", "w1s", "w2", "w2s", "ws", "out")],
    *[({n: ODD}, INVALID) for n in ("x", "xs", "idx", "wt", "w1", "w1s", "w2", "w2s", "ws", "out")],
    (dict(dt=0), INVALID), (dict(dt=1), INVALID), (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(K=17), INVALID),
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(begin=-1), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID),
    (dict(n=16), INVALID), (dict(out=A[0]), INVALID), (dict(out=ctypes.c_void_p(0x10000 + 512)), INVALID), (dict(T=65), UNSUPPORTED), (dict(H=192), UNSUPPORTED), (dict(I=64), UNSUPPORTED),
    (dict(H=1 << 16), UNSUPPORTED), (dict(I=1 << 16), UNSUPPORTED)], ids=str)
def test_decode_refuses(lib, kw, rc):
    assert decode(lib, **kw) == rc


def test_decode_of_no_rows(lib):
    assert decode(lib, T=0, x=None, xs=None, idx=None, wt=None, ws=None, out=None, n=0) == OK
    for f in ((0, 2, 128), (65, 2, 128), (4, 0, 128), (4, 17, 128), (4, 2, 64), (4, 2, 0)):
        assert lib.moe_expert_ffn_decode_workspace_bytes(*f) == 0
    assert lib.moe_expert_ffn_decode_workspace_bytes(4, 2, 128) >= 4 * 2 * (128 + 4)


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    l = torch.zeros(2, 8)
    i = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_rmsnorm(x, x[0], 1e-6, x)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_rmsnorm_backward(x, x, x[0], l[:, 0], x)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_router_topk(l, i, torch.zeros(2, 2))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_router_topk_backward(torch.zeros(2, 2), l, i, l)


def test_router_config_refuses_unknown_scores():
    with pytest.raises(ValueError):
        moe.RouterConfig(score="relu").c()
    c = moe.RouterConfig(score="sigmoid", groups=4, topk_groups=2, group_top=2, scale=2.5, normalize=False).c()
    assert (c.score, c.normalize, c.groups, c.topk_groups, c.group_top, c.scale) == (1, 0, 4, 2, 2, 2.5)

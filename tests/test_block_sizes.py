"""Sizes past int32, which the C ABI cannot be told: the binding refuses them, instead of working on what is left of the number
(2^32 + 4 rows as 4). No GPU and no memory: tensors of the "meta" device, and nothing may be launched."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from combine_moe_dispatch_02_amd import block

BIG = 2 ** 32 + 4
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def t(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture(autouse=True)
def nothing_is_launched(monkeypatch):
    def launch(name, *a):
        raise AssertionError(f"{name} was launched")

    monkeypatch.setattr(block, "_device", lambda x, name: x.get_device())
    monkeypatch.setattr(block, "_launch", launch)


def plan(T, K, E, tile):
    return moe.Plan(T, K, 0, E, tile, 4 * tile, *(t(4, dtype=I32) for _ in range(7)))


class Ws:
    buf, nbytes = t(64, dtype=U8), 64


CALLS = {
    "norm rows": lambda: moe.moe_rmsnorm(t(BIG, 8), t(8), 1e-6, t(BIG, 8)),
    "norm width": lambda: moe.moe_rmsnorm(t(1, BIG), t(BIG), 1e-6, t(1, BIG)),
    "norm backward": lambda: moe.moe_rmsnorm_backward(t(BIG, 8), t(BIG, 8), t(8), t(BIG, dtype=F32), t(BIG, 8)),
    "router": lambda: moe.moe_router_topk(t(BIG, 1), t(BIG, 1, dtype=I32), t(BIG, 1, dtype=F32)),
    "router experts": lambda: moe.moe_router_topk(t(1, BIG), t(1, 1, dtype=I32), t(1, 1, dtype=F32)),
    "router backward": lambda: moe.moe_router_topk_backward(t(BIG, 1, dtype=F32), t(BIG, 1), t(BIG, 1, dtype=I32), t(BIG, 1)),
    "dispatch pool": lambda: moe.moe_dispatch_quantized(t(1, 128, dtype=U8), t(1, 1, dtype=F32), plan(1, 1, 1, 16), t(BIG, 128, dtype=U8),
                                                        t(BIG, 1, dtype=F32), 1, Ws, "fp8"),
    "dispatch epoch": lambda: moe.moe_dispatch_quantized(t(1, 128, dtype=U8), t(1, 1, dtype=F32), plan(1, 1, 1, 16), t(64, 128, dtype=U8),
                                                         t(64, 1, dtype=F32), 2 ** 32 + 1, Ws, "fp8"),
    "decode begin": lambda: moe.moe_expert_ffn_decode(t(1, 128), None, t(1, 1, dtype=I32), t(1, 1, dtype=F32), t(1, 256, 64, dtype=U8),
                                                      t(1, 256, 4, dtype=U8), t(1, 128, 64, dtype=U8), t(1, 128, 4, dtype=U8),
                                                      t(512, dtype=U8), t(1, 128), expert_begin=2 ** 32),
    "norm workspace": lambda: moe.rmsnorm_backward_workspace_bytes(BIG, 8),
    "decode workspace": lambda: moe.expert_ffn_decode_workspace_bytes(BIG, 1, 128),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(name):
    with pytest.raises(ValueError, match="past 2"):
        CALLS[name]()


def test_int32_max_is_a_size():
    with pytest.raises(AssertionError, match="moe_router_topk was launched"):
        n = 2 ** 31 - 1
        moe.moe_router_topk(t(n, 1), t(n, 1, dtype=I32), t(n, 1, dtype=F32))

"""What Adapters, AdapterRows and StreamMoE's use of them refuse, before anything is enqueued."""
from types import SimpleNamespace

import pytest
import torch

import combine_moe_dispatch_02_amd as moe

BF16 = torch.bfloat16


def pair(n=2, R=8, K=64, N=64):
    return torch.zeros(n, R, K, dtype=BF16), torch.zeros(n, N, R, dtype=BF16)


def test_rows():
    rows = moe.AdapterRows(4, 2, device="cpu")
    assert rows.plan is None                                 # up to 64 rows are found by their ids
    with pytest.raises(RuntimeError, match="set"):
        rows.by()
    for bad in (torch.zeros(4), torch.zeros(5, dtype=torch.int32), torch.zeros(4, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="ids"):
            rows.set(bad)
    ids = torch.zeros(4, dtype=torch.int32)
    assert rows.set(ids).by() == {"ids": ids, "id_begin": 0}
    assert moe.AdapterRows(65, 2, device="cpu").plan is not None
    assert moe.AdapterRows(1, 2, train=True, device="cpu").plan is not None


def test_tiles():
    assert [moe.adapter_tile(T, n) for T, n in ((1, 1), (2047, 1), (2048, 1), (2999, 1), (3000, 1), (6399, 100), (6400, 100))] == [
        16, 16, 32, 32, 128, 32, 128]


def test_no_rows():
    rows = moe.AdapterRows(0, 2, train=True, device="cpu")
    assert rows.plan is None
    ad = moe.Adapters(*pair(), rows, train=True)
    assert ad.v.shape == (0, 8) and ad.da.shape == (2, 8, 64) and ad.db.shape == (2, 64, 8)


def test_tables():
    a, b = pair()
    rows = moe.AdapterRows(4, 2, device="cpu")
    for bad in ((a[0], b), (a, b[:1]), (a[:, :4], b)):
        with pytest.raises(ValueError, match="must be"):
            moe.Adapters(*bad, rows)
    with pytest.raises(ValueError, match="rows are of"):
        moe.Adapters(a, b, moe.AdapterRows(4, 3, device="cpu"))
    with pytest.raises(ValueError, match="train"):
        moe.Adapters(a, b, rows, train=True)
    for train in (False, True):
        ad = moe.Adapters(a, b, moe.AdapterRows(4, 2, train=train, device="cpu"), train=train)
        with pytest.raises(RuntimeError, match="add"):
            ad.backward(torch.zeros(4, 64, dtype=BF16), None)


def test_layer():
    layer = SimpleNamespace(H=64)
    check = lambda ad, x, ax=None: moe.StreamMoE._check_adapters(layer, ad, x, ax)  # noqa: E731
    x, quantised = torch.zeros(4, 64, dtype=BF16), (torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    ad = moe.Adapters(*pair(), moe.AdapterRows(4, 2, device="cpu"))
    check(None, quantised)
    check(ad, x)
    check(ad, quantised, x)
    for rows in ((quantised,), (x.float(),), (quantised, x.float())):
        with pytest.raises(ValueError, match="bf16 rows"):
            check(ad, *rows)
    for other in (pair(K=32), pair(N=32)):
        with pytest.raises(ValueError, match="do not match"):
            check(moe.Adapters(*other, ad.rows), x)
    with pytest.raises(ValueError, match="do not match"):
        check(ad, x[:3])

"""Which batch a backward pass belongs to: gradients are refused where the rows were grouped anew, or an add failed, since the
add they are of. The kernels' calls are replaced: no GPU."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from combine_moe_dispatch_02_amd import adapters as module

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """What would be launched, in order."""
    log = []
    monkeypatch.setattr(module, "moe_plan", lambda ids, *a: log.append("plan"))
    monkeypatch.setattr(module, "moe_adapter", lambda x, *a, **k: log.append("add"))
    monkeypatch.setattr(module, "moe_adapter_backward", lambda dout, x, *a, **k: log.append(x))
    return log


def make(T=4, n=2, R=8, K=64, N=64, count=1):
    rows = moe.AdapterRows(T, n, train=True, device="cpu")
    table = lambda: (torch.zeros(n, R, K, dtype=BF16), torch.zeros(n, N, R, dtype=BF16))  # noqa: E731
    return rows, [moe.Adapters(*table(), rows, train=True) for _ in range(count)]


def ids(T=4, e=0):
    return torch.full((T,), e, dtype=torch.int32)


def batch(T=4):
    return torch.zeros(T, 64, dtype=BF16), torch.zeros(T, 64, dtype=BF16)


def test_rows_grouped_anew_between_add_and_backward(calls):
    rows, (one, two) = make(count=2)
    (x, out), dout = batch(), batch()[0]
    rows.set(ids())
    one.add(x, out), two.add(x, out)
    two.backward(dout, None)                      # several projections share a grouping
    rows.set(ids(e=1))                            # the next batch
    before = list(calls)
    for late in (one, two):
        with pytest.raises(RuntimeError, match="set"):
            late.backward(dout, None)
        with pytest.raises(RuntimeError, match="set"):
            late.check_backward()
    assert calls == before                        # nothing was launched
    two.add(x, out)
    two.backward(dout, None)
    with pytest.raises(RuntimeError, match="set"):
        one.backward(dout, None)


def test_gradients_twice_of_one_add(calls):
    rows, (ad,) = make()
    rows.set(ids())
    x, out = batch()
    ad.add(x, out)
    ad.backward(out, None)
    ad.backward(out, None)
    assert calls[-1] is x and calls[-2] is x


def test_an_add_that_failed_leaves_the_last_ones_batch(calls, monkeypatch):
    rows, (ad,) = make()
    rows.set(ids())
    (x, out), (other, _) = batch(), batch()
    ad.add(x, out)

    def fail(*a, **k):
        raise ValueError("refused")
    monkeypatch.setattr(module, "moe_adapter", fail)
    with pytest.raises(ValueError):
        ad.add(other, out)
    ad.backward(out, None)
    assert calls[-1] is x


def test_a_set_that_failed_leaves_the_grouping(calls, monkeypatch):
    rows, (ad,) = make()
    first = ids()
    rows.set(first)
    x, out = batch()
    ad.add(x, out)

    def fail(*a, **k):
        raise ValueError("refused")
    monkeypatch.setattr(module, "moe_plan", fail)
    with pytest.raises(ValueError):
        rows.set(ids(e=1))
    assert rows.ids is first
    ad.backward(out, None)
    assert calls[-1] is x


def test_rows_are_grouped_on_their_own_device(calls, monkeypatch):
    """Not on the current one: moe_plan launches on whatever device is current, on its current stream."""
    rows, _ = make()
    inside = []

    class DeviceOf:
        def __init__(self, t):
            self.t = t

        def __enter__(self):
            inside.append(self.t)

        def __exit__(self, *a):
            inside.append(None)

    monkeypatch.setattr(torch.cuda, "device_of", DeviceOf)
    monkeypatch.setattr(module, "moe_plan", lambda t, *a: calls.append(inside[-1] if inside else None))
    mine = ids()
    rows.set(mine)
    assert calls[-1] is not None and calls[-1].data_ptr() == mine.data_ptr() and inside[-1] is None
    with pytest.raises(ValueError, match="device"):
        rows.set(torch.empty(4, dtype=torch.int32, device="meta"))
    assert len(calls) == 1

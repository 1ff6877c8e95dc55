"""What StreamMoE refuses of adapters before it enqueues anything, and that its streams are joined where adding them fails. The kernels'
calls are replaced: no GPU."""
from types import SimpleNamespace

import pytest
import torch

import combine_moe_dispatch_02_amd as moe
from combine_moe_dispatch_02_amd import adapters as adapters_module, block as block_module, layer as layer_module

BF16 = torch.bfloat16
H, K = 64, 2


class Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")

    def wait_event(self, event):
        pass


@pytest.fixture
def log(monkeypatch):
    calls = []
    note = lambda name: lambda *a, **k: calls.append(name)  # noqa: E731
    for name in ("moe_plan", "moe_dispatch", "moe_expert_ffn", "moe_expert_ffn_train", "moe_expert_ffn_combine", "moe_combine",
                 "moe_combine_backward", "moe_expert_ffn_backward", "moe_dispatch_backward", "device_cu_count"):
        monkeypatch.setattr(layer_module, name, note(name))
    monkeypatch.setattr(layer_module.StreamMoE, "_concurrent_cfg", lambda self: None)
    monkeypatch.setattr(block_module, "moe_expert_ffn_decode", note("moe_expert_ffn_decode"))
    monkeypatch.setattr(adapters_module, "moe_plan", lambda *a: None)
    monkeypatch.setattr(adapters_module, "moe_adapter", note("add"))
    monkeypatch.setattr(adapters_module, "moe_adapter_backward", note("adapter gradients"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream("cur", calls))
    monkeypatch.setattr(torch.cuda, "Event", lambda: SimpleNamespace(record=lambda s: None))
    return calls


def make_layer(T=4, train=False, on_completion=False, dtype="bf16"):
    layer = object.__new__(moe.StreamMoE)
    e = torch.empty(T, H, dtype=BF16)
    vars(layer).update(T=T, H=H, I=64, K=K, E_local=2, expert_begin=0, dtype=dtype, train=train, combine_on_completion=on_completion,
                       plan=None, ws=None, pool=None, pool_s=None, y_pool=None, g_pool=None, dx_pool=None, dw=None, cfg=None, epoch=0,
                       decode_ws=None, out=e, dx=e.clone(), _added=None)
    return layer


def make_adapters(T=4, train=False, set_rows=True):
    rows = moe.AdapterRows(T, 2, train=train, device="cpu")
    if set_rows:
        rows.set(torch.zeros(T, dtype=torch.int32))
    return moe.Adapters(torch.zeros(2, 8, H, dtype=BF16), torch.zeros(2, H, 8, dtype=BF16), rows, train=train)


def inputs(T=4):
    return torch.zeros(T, H, dtype=BF16), torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(2, 1), torch.zeros(2, 1)


def streams(log):
    return Stream("compute", log), Stream("comm", log)


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("train,on_completion", [(False, False), (True, False), (False, True)])
def test_forward_refuses_before_it_enqueues(log, two, train, on_completion):
    layer = make_layer(train=train, on_completion=on_completion)
    st = streams(log) if two else None
    wide = torch.zeros(5, H, dtype=BF16)
    with pytest.raises(ValueError, match="do not match"):           # 5 rows' adapters beside the layer's 4
        layer.forward(*inputs(), streams=st, adapters=make_adapters(5), adapter_x=wide)
    with pytest.raises(RuntimeError, match="set"):
        layer.forward(*inputs(), streams=st, adapters=make_adapters(set_rows=False))
    assert not log and layer.epoch == 0
    layer.forward(*inputs(), streams=st, adapters=make_adapters())
    assert "add" in log


def test_decode_refuses_before_it_enqueues(log):
    layer = make_layer(dtype="mxfp4")
    few = [t[:3] for t in inputs()[:3]]
    for ad, x in ((make_adapters(4), inputs()[0]), (make_adapters(2), inputs(2)[0])):
        with pytest.raises(ValueError, match="do not match"):
            layer.decode(*few, *inputs()[3:], None, None, adapters=ad, adapter_x=x)
    with pytest.raises(RuntimeError, match="set"):
        layer.decode(*few, *inputs()[3:], None, None, adapters=make_adapters(3, set_rows=False))
    assert not log
    layer.decode(*few, *inputs()[3:], None, None, adapters=make_adapters(3))
    assert log == ["moe_expert_ffn_decode", "add"]


@pytest.mark.parametrize("train,on_completion", [(False, False), (True, False), (False, True)])
def test_streams_are_joined_where_adapters_fail(log, monkeypatch, train, on_completion):
    def fail(*a, **k):
        raise ValueError("on another device")
    layer, ad = make_layer(train=train, on_completion=on_completion), make_adapters(train=train)
    if train:
        layer.forward(*inputs(), streams=streams(log), adapters=ad)
        monkeypatch.setattr(adapters_module, "moe_adapter_backward", fail)
        del log[:]
        with pytest.raises(ValueError, match="another device"):
            layer.backward(inputs()[0], *inputs()[2:], streams=streams(log), adapters=ad)
        assert log[-1] == "cur waits for comm"
    monkeypatch.setattr(adapters_module, "moe_adapter", fail)
    del log[:]
    with pytest.raises(ValueError, match="another device"):
        layer.forward(*inputs(), streams=streams(log), adapters=ad)
    assert log[-1] == "cur waits for comm" and (not on_completion or "cur waits for compute" in log)


def backward(layer, ad=None, st=None):
    return layer.backward(inputs()[0], *inputs()[2:], streams=st, adapters=ad)


@pytest.mark.parametrize("two", [False, True])
def test_backward_takes_the_adapters_of_the_last_forward(log, two):
    layer, ad, other = make_layer(train=True), make_adapters(train=True), make_adapters(train=True)
    st = streams(log) if two else None
    for a in (ad, other):
        a.add(*2 * [inputs()[0]])                 # each has a batch of its own
    with pytest.raises(RuntimeError, match="last forward"):
        backward(layer, ad, st)                   # no forward at all
    layer.forward(*inputs(), streams=st, adapters=ad)
    del log[:]
    with pytest.raises(RuntimeError, match="last forward"):
        backward(layer, other, st)
    assert not log
    backward(layer, ad, st)
    backward(layer, None, st)                     # their share left out, to be taken by hand
    ad.add(*2 * [inputs()[0]])                    # something else since: v is of that
    with pytest.raises(RuntimeError, match="last forward"):
        backward(layer, ad, st)
    layer.forward(*inputs(), streams=st, adapters=ad)
    layer.forward(*inputs(), streams=st)          # without
    with pytest.raises(RuntimeError, match="last forward"):
        backward(layer, ad, st)


def test_backward_refuses_the_gradient_of_other_rows_than_the_layers(log):
    layer, ad = make_layer(train=True), make_adapters(train=True)
    layer.forward(*inputs(), adapters=ad, adapter_x=inputs()[0])
    with pytest.raises(RuntimeError, match="adapter_x"):
        backward(layer, ad)                       # one dx cannot be that of two inputs
    backward(layer)
    x, *more = inputs()
    layer.forward(x, *more, adapters=ad, adapter_x=x[:])
    backward(layer, ad)


def test_backward_refuses_where_the_adapters_of_the_last_forward_failed(log, monkeypatch):
    layer, ad = make_layer(train=True), make_adapters(train=True)
    layer.forward(*inputs(), adapters=ad)

    def fail(*a, **k):
        raise ValueError("refused")
    monkeypatch.setattr(adapters_module, "moe_adapter", fail)
    with pytest.raises(ValueError):
        layer.forward(*inputs(), adapters=ad)
    with pytest.raises(RuntimeError, match="last forward"):
        backward(layer, ad)


@pytest.mark.parametrize("two", [False, True])
def test_rows_that_the_layer_overwrites_before_the_adapters_read_them(log, two):
    """forward() without adapters takes the layer's own out as x; adapters would read what it has become."""
    layer, ad = make_layer(train=True), make_adapters(train=True)
    st = streams(log) if two else None
    x, *more = inputs()
    wide = torch.empty(4, 2 * H, dtype=BF16)
    layer.out = wide[:, :H]
    layer.forward(layer.out, *more, streams=st)
    del log[:]
    for rows, other in ((layer.out, None), (x, layer.out), (x, wide[:, 8:8 + H])):
        with pytest.raises(ValueError, match="overlap"):
            layer.forward(rows, *more, streams=st, adapters=ad, adapter_x=other)
    assert not log
    layer.forward(x, *more, streams=st, adapters=ad)
    with pytest.raises(ValueError, match="overlap"):
        layer.backward(layer.dx, *inputs()[2:], streams=st, adapters=ad)
    layer.backward(layer.dx, *inputs()[2:], streams=st)
    decoder = make_layer(dtype="mxfp4")
    with pytest.raises(ValueError, match="overlap"):
        decoder.decode(x, *more, None, None, adapters=make_adapters(), adapter_x=decoder.out)
    few = [t[:2] for t in (x, *more[:2])]
    decoder.decode(*few, *more[2:], None, None, adapters=make_adapters(2), adapter_x=decoder.out[2:])

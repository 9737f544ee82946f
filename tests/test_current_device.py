"""The binding works on its tensors' device, whichever device is current (host
side: the devices are stand-ins)."""
import contextlib
import inspect
import types

import pytest
import torch

import grouped_top_routing_amd as gtr
from grouped_top_routing_amd import _lib as L

CALLS = ("route", "route_replay", "permute", "expert_ffn", "expert_gate_up", "expert_down",
         "combine", "layer_forward", "layer_forward_noalloc", "layer_forward_fp8",
         "layer_forward_lora", "pack_weights", "quantize_fp8", "expert_ffn_fp8",
         "expert_gate_up_fp8", "expert_down_fp8", "expert_ffn_lora")


@pytest.fixture
def current(monkeypatch):
    """Two devices; the value is the current one's number, [0] at first."""
    now = [0]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return now


def _tensor(index):
    return types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", index))


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_with_their_tensors_device_current(current, index):
    seen = L._on_their_device(lambda *a, **kw: (a, kw, current[0]))
    t = _tensor(index)
    assert seen(t, 3, b=4) == ((t, 3), {"b": 4}, index) and current == [0]
    assert seen(None, w=t) == ((None,), {"w": t}, index) and current == [0]
    assert seen(torch.zeros(1), 2)[2] == 0  # a host tensor: the call's own checks refuse it


@pytest.mark.parametrize("name", CALLS)
def test_every_call_does(name):
    fn = getattr(gtr, name)
    assert inspect.unwrap(fn) is not fn and inspect.unwrap(fn).__name__ == name


def test_capture_is_looked_for_on_the_tensors_device(current, monkeypatch):
    capturing = {0: True, 1: False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[current[0]])
    assert L._capturing(torch.device("cuda", 0)) is True
    assert L._capturing(torch.device("cuda", 1)) is False
    assert current == [0]


def test_adamw_asks_for_its_own_device(monkeypatch):
    """A graph captured on another device is no business of this optimizer's."""
    asked = []

    def capturing(device):
        asked.append(device)
        return True

    monkeypatch.setattr(L, "_capturing", capturing)
    opt = gtr.AdamW.__new__(gtr.AdamW)
    opt.params, opt._rows, opt.lr = (), (), 1e-3
    opt.device, opt._opt, opt._step_dev, opt._steps = torch.device("cuda", 1), L.MoeAdamw(), None, 0
    with pytest.raises(RuntimeError, match="capturable"):
        opt.step([])
    assert asked == [torch.device("cuda", 1)]

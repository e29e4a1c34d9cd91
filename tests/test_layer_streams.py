"""Which stream a layer operator runs on, without a GPU: torch's streams are
stood in for by objects with a handle."""

import pytest
import torch

from matrix_optimizer_step_muon_amd import layer


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream

    __hash__ = None


class Memory:
    """Stands in for a tensor: which streams it was recorded on."""

    def __init__(self):
        self.on = []

    def record_stream(self, stream):
        self.on.append(stream.cuda_stream)


@pytest.fixture
def current(monkeypatch):
    """Sets the current stream's handle."""
    now = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(now[0]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: now[0], raising=False)
    # what torch does with a handle: 0 gives a stream of its pool
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a: Stream(handle or 0xBAD))

    def to(handle):
        now[0] = handle
    return to


def ran_on(monkeypatch, stream):
    """The handle that a WGrad hands the library for run(stream)."""
    seen = []

    class Lib:
        def muon_wgrad(self, items, n, dtype, g_dtype, ws, ws_bytes, handle):
            seen.append(handle)
            return 0

    monkeypatch.setattr(layer, "lib", Lib)
    plan = object.__new__(layer.WGrad)
    plan._items, plan._n, plan._dtype, plan._gdtype = None, 1, 1, 1
    plan._tensors, plan.workspace = [Memory()], torch.empty(16, dtype=torch.uint8)
    plan.run(stream)
    return seen[0]


@pytest.mark.parametrize("now", [0, 7])
def test_a_raw_handle_names_that_stream(current, monkeypatch, now):
    current(now)
    for handle in (0, 7, 9):
        assert ran_on(monkeypatch, handle) == handle
        assert ran_on(monkeypatch, Stream(handle)) == handle
    assert ran_on(monkeypatch, None) == now

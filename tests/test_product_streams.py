"""Which stream the gated block and the 8-bit products run on, and on which their
memory is recorded, without a GPU."""

import pytest
import torch

from matrix_optimizer_step_muon_amd import layer
from test_layer_streams import Stream, q8, world  # noqa: F401  (a fixture)


@pytest.fixture
def on_cpu(world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch, "device", lambda *a, real=torch.device: real("cpu"))
    return world


def mlp():
    x, wg, wu, wd = torch.zeros(40, 64), torch.zeros(96, 64), torch.zeros(96, 64), torch.zeros(64, 96)
    m = layer.GatedMLP(x, wg, wu, wd, saved=tuple(q8(40, 96) for _ in range(3)))
    assert m.workspace.numel() > 0
    return m, {t.data_ptr() for t in (x, wg, wu, wd, m.y, m.d_x, m.d_a, m.d_b, m.workspace)} | {
        t.data_ptr() for q in (m.a, m.b, m.s) for t in (q.q, q.e)}


def linear(on_cpu):
    x = layer.Q8(40, 64, "e4m3", q=torch.zeros(40, 64, dtype=torch.uint8), e=torch.zeros(40, 2, dtype=torch.uint8))
    w, y, c = layer.W8(96, 64), torch.zeros(40, 96), torch.zeros(40, 96)
    p = layer.Linear8([(x, w, y, 1.0, c)])
    return p, {t.data_ptr() for t in (x.q, x.e, w.q, w.qt, w.e, y, c, p.workspace)}, w


@pytest.mark.parametrize("now", [0, 7])
def test_a_raw_handle_names_that_stream(on_cpu, now):
    on_cpu.now = now
    m, _ = mlp()
    p, _, w = linear(on_cpu)
    for handle in (0, 7, 9):
        for stream in (handle, Stream(handle)):
            m.forward(stream), m.backward(torch.zeros(40, 64), stream), p.run(stream)
            layer.w8_save(torch.zeros(96, 64), w, stream), layer.w8_load(w, torch.zeros(96, 64), stream)
            assert on_cpu.launched == [handle] * 5
            on_cpu.launched.clear()
    m.forward()
    assert on_cpu.launched == [now]
    assert not on_cpu.on(0xBAD)


def test_the_current_stream_is_recorded_on_all_memory_that_the_object_holds(on_cpu):
    (m, memory), (p, tensors, w) = mlp(), linear(on_cpu)
    on_cpu.now = 7
    m.forward()
    assert on_cpu.on(7) == memory
    on_cpu.now = 8
    m.backward(torch.zeros(40, 64))
    assert on_cpu.on(8) >= memory
    on_cpu.now = 9
    p.run()
    assert on_cpu.on(9) == tensors
    on_cpu.now = 10
    layer.w8_save(torch.zeros(96, 64), w)
    assert on_cpu.on(10) == {t.data_ptr() for t in w.tensors()}
    on_cpu.now = 11
    layer.w8_load(w, torch.zeros(96, 64))
    assert on_cpu.on(11) == {t.data_ptr() for t in w.tensors()}


def test_a_named_stream_is_recorded_on_the_calls_own_tensors(on_cpu):
    m, _ = mlp()
    dy, w, x = torch.zeros(40, 64), layer.W8(96, 64), torch.zeros(96, 64)
    m.backward(dy, 5)
    assert dy.data_ptr() in on_cpu.on(5)
    layer.w8_save(x, w, Stream(6))
    assert on_cpu.on(6) == {t.data_ptr() for t in w.tensors()} | {x.data_ptr()}


def test_another_current_device_is_refused(on_cpu, monkeypatch):
    (m, _), (p, _, _) = mlp(), linear(on_cpu)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (m.forward, p.run):
        with pytest.raises(layer.MuonError, match="cuda:0"):
            call()
    assert not on_cpu.launched
    monkeypatch.undo()


def test_checkpoints_and_weights_elsewhere_are_refused(on_cpu, monkeypatch):
    """What holds no device tensors of the current device."""
    def matrix(t, name, *a, **k):
        if t.data_ptr() in away:
            raise layer.MuonError(-1, f"{name} is elsewhere")
        return t
    x = q8(40, 64)
    x8 = layer.Q8(40, 64, "e4m3", q=x.q, e=x.e)
    w, y = layer.W8(96, 64), torch.zeros(40, 96)
    a, b = q8(40, 96), q8(40, 96)
    t = [torch.zeros(40, 64), torch.zeros(96, 64), torch.zeros(96, 64), torch.zeros(64, 96)]
    monkeypatch.setattr(layer, "_matrix", matrix)
    for bad, call in ((x.q, lambda: layer.Linear8([(x8, w, y)])), (w.q, lambda: layer.Linear8([(x8, w, y)])),
                      (b.q, lambda: layer.GatedMLP(*t, saved=(a, b))), (w.q, lambda: layer.w8_save(t[1], w)),
                      (w.q, lambda: layer.w8_load(w, t[1]))):
        away = {bad.data_ptr()}
        with pytest.raises(layer.MuonError, match="elsewhere"):
            call()

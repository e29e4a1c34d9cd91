"""Which stream a layer operator runs on, and on which its memory is recorded,
without a GPU: torch's streams are stood in for by objects with a handle, and
the library's launches by a note of the handle they were given."""

import pytest
import torch

from matrix_optimizer_step_muon_amd import layer, muon


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream

    __hash__ = None

    def __enter__(self):
        self.before, self.world.now = self.world.now, self.cuda_stream

    def __exit__(self, *a):
        self.world.now = self.before


class World:
    def __init__(self):
        self.now = 0            # the current stream
        self.launched = []      # handles
        self.recorded = set()   # (address, handle)

    def on(self, handle):
        return {p for p, h in self.recorded if h == handle}


@pytest.fixture
def world(monkeypatch):
    w, real = World(), muon.lib()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(w.now))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s or Stream(w.now))
    monkeypatch.setattr(Stream, "world", w, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: w.now, raising=False)
    # what torch does with a handle: 0 gives a stream of its pool
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a: Stream(handle or 0xBAD))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.recorded.add((t.data_ptr(), s.cuda_stream)))

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_workspace"):
                return getattr(real, name)

            def launch(*args):
                w.launched.append(args[-1])
                return 0
            return launch

    monkeypatch.setattr(layer, "lib", Lib)
    monkeypatch.setattr(layer, "_matrix", lambda t, *a, **k: t)
    return w


def q8(rows, cols):
    return layer.Q8(rows, cols, q=torch.zeros(rows, cols, dtype=torch.uint8), e=torch.zeros(rows, cols // 32, dtype=torch.uint8))


def plan():
    """A WGrad, and the addresses of all the memory it uses."""
    dy, x, g, s = torch.zeros(5000, 320), q8(5000, 64), torch.zeros(320, 64), torch.zeros(64)
    p = layer.WGrad([(dy, x, g, s)])
    assert p.workspace.numel() > 0
    return p, {t.data_ptr() for t in (dy, x.q, x.e, g, s, p.workspace)}


def site():
    x, w = torch.zeros(4, 64), torch.zeros(64)
    s = layer.NormSite(x, torch.zeros(4, 64), w, w_post=torch.zeros(64), saved=(q8(4, 64), q8(4, 64), torch.zeros(4), torch.zeros(4)))
    return s, [s.branch, s.residual, s.w_pre, s.w_post, s.y, s.h, s.rstd_y, s.rstd_b, s.u.q, s.u.e, s.v.q, s.v.e]


@pytest.mark.parametrize("now", [0, 7])
def test_a_raw_handle_names_that_stream(world, now):
    world.now = now
    p, _ = plan()
    s, _ = site()
    for handle in (0, 7, 9):
        for stream in (handle, Stream(handle)):
            p.run(stream), s.forward(stream), s.backward(None, torch.zeros(4, 64), stream)
            assert world.launched == [handle] * 3
            world.launched.clear()
    p.run()
    assert world.launched == [now]
    assert not world.on(0xBAD)


def test_the_current_stream_is_recorded_on_all_memory_that_the_object_holds(world):
    # Inside `with torch.cuda.stream(side)`: dropping the object afterwards must
    # not hand its buffers out before side is done with them.
    (p, memory), (s, tensors), ckpt, x = plan(), site(), q8(4, 64), torch.zeros(4, 64)
    world.now = 7
    p.run()
    assert world.on(7) == memory
    world.now = 8
    s.forward()
    assert world.on(8) == {t.data_ptr() for t in tensors}
    world.now = 9
    layer.q8_save(x, ckpt)
    assert world.on(9) == {ckpt.q.data_ptr(), ckpt.e.data_ptr()}
    world.now = 10
    layer.q8_load(ckpt, x)
    assert world.on(10) == {ckpt.q.data_ptr(), ckpt.e.data_ptr()}


def test_gradients_made_on_one_stream_are_recorded_on_the_others_that_use_them(world):
    s, tensors = site()
    dh = torch.zeros(4, 64)
    s.backward(None, dh, Stream(7))
    made = [s.d_residual, s.d_branch, s.d_w_pre, s.d_w_post, s._workspace]
    assert world.on(7) >= {t.data_ptr() for t in tensors + [dh]}
    s.backward(None, dh)
    assert world.on(0) == {t.data_ptr() for t in made}
    world.now = 3
    s.forward()
    assert world.on(3) == {t.data_ptr() for t in tensors}
    s.backward(None, dh)
    assert world.on(3) == {t.data_ptr() for t in tensors + made}


def test_a_named_stream_is_recorded_on_the_calls_own_tensors(world):
    s, tensors = site()
    for dy in (None, torch.zeros(4, 64)):
        dh = torch.zeros(4, 64)
        s.backward(dy, dh, 5)
        assert {t.data_ptr() for t in (dy, dh) if t is not None} <= world.on(5)
    ckpt, x = q8(4, 64), torch.zeros(4, 64)
    layer.q8_save(x, ckpt, Stream(6))
    assert world.on(6) == {ckpt.q.data_ptr(), ckpt.e.data_ptr(), x.data_ptr()}


def test_a_stream_is_recorded_once_and_the_first_one_never(world):
    p, memory = plan()
    for expected in (memory, set()):
        for world.now in (0, 7):
            p.run()
        assert not world.on(0) and world.on(7) == expected
        world.recorded.clear()

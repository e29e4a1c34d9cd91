"""The gated block and the 8-bit products captured into HIP graphs and replayed, with
eager work between; and buffers of objects dropped while another stream works on
them."""

import numpy as np
import pytest

from layer_helpers import dev, rng, say
from matrix_optimizer_step_muon_amd import layer
from product_helpers import Mlp
from test_layer_streams_gpu import keep_busy

pytestmark = pytest.mark.gpu


def bits(ts):
    import torch
    torch.cuda.synchronize()
    return [t.clone() for t in ts]


def same(got, want):
    import torch
    torch.cuda.synchronize()
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def checkpoint(seed, rows, cols):
    """Random rows as an e4m3 checkpoint."""
    return layer.q8_save(dev(rng(seed).standard_normal((rows, cols)), "f32"), layer.Q8(rows, cols, "e4m3"))


class Step:
    """What a training step does around its weights in 8 bits."""

    def __init__(self, rows, width, inner, dtype, kind, seed):
        self.m = Mlp(rows, width, inner, width, dtype, "silu", kind, seed=seed)
        m = self.m.mlp
        self.w8 = layer.W8(inner, width)
        q = checkpoint(seed, rows, width)
        self.out = [dev(np.zeros((rows, n)), dtype) for n in (inner, width)]
        back = checkpoint(seed + 1, rows, inner)
        self.products = [layer.Linear8([(q, self.w8, self.out[0])]), layer.Linear8([(back, self.w8, self.out[1])], transposed=True)]
        self.results = [m.y, m.a.q, m.b.q, m.s.q, m.d_a, m.d_b, m.d_x, *self.w8.tensors(), *self.out]

    def run(self):
        self.m.forward().backward()
        layer.w8_save(self.m.mlp.w_up, self.w8)
        for p in self.products:
            p.run()

    def change(self, k):
        self.m.mlp.x.mul_(0.5 + k)
        self.m.mlp.w_up.mul_(1.5 - 0.25 * k)

    def spoil(self):
        for t in self.results:
            t.zero_()


def capture(f):
    import torch
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        f()
    return g


SHAPES = [(3, 200, 264, "bf16", "int8"), (16, 64, 96, "f32", "e4m3"), (300, 136, 520, "bf16", "e4m3"), (129, 77, 130, "f32", "int8")]


@pytest.mark.parametrize("rows,width,inner,dtype,kind", SHAPES)
def test_captured_and_replayed(rows, width, inner, dtype, kind):
    say(rows, width, inner, dtype, kind)
    s = Step(rows, width, inner, dtype, kind, 1)
    s.run()                                   # eager, before anything is captured
    want = bits(s.results)
    s.spoil()
    g = capture(s.run)
    assert not any(bool(t.any()) for t in bits(s.results)), "capture must not run it"
    for k in range(4):
        g.replay()
        assert same(s.results, want), k
        s.change(k)                           # and an eager pass between the replays
        s.run()
        want = bits(s.results)
        s.spoil()


def test_two_graphs_of_the_same_objects():
    """They share the objects' workspaces and follow each other on one stream."""
    s = Step(300, 136, 520, "bf16", "int8", 2)
    s.run()
    want = bits(s.results)
    forward = capture(s.m.forward)
    rest = capture(lambda: (s.m.backward(), layer.w8_save(s.m.mlp.w_up, s.w8), [p.run() for p in s.products]))
    for k in range(3):
        s.spoil()
        forward.replay()
        rest.replay()
        assert same(s.results, want), k


def test_two_graphs_on_two_streams_at_once():
    """Of objects with workspaces of their own."""
    import torch
    steps = [Step(40 + 300 * i, 200, 1032, "bf16", "int8", 4 + i) for i in range(2)]
    wants = []
    for s in steps:
        s.run()
        wants.append(bits(s.results))
        s.spoil()
    graphs = [capture(s.run) for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    assert all(same(s.results, w) for s, w in zip(steps, wants))


def test_products_run_on_an_ambient_stream_and_dropped():
    import torch
    g = rng(5)
    x, w = checkpoint(5, 40, 20000), layer.W8(64, 20000)
    layer.w8_save(dev(g.standard_normal((64, 20000)), "bf16"), w)
    y, want = (dev(np.zeros((40, 64)), "bf16") for _ in range(2))
    layer.Linear8([(x, w, want)]).run()
    plan = layer.Linear8([(x, w, y)])
    address, size = plan.workspace.data_ptr(), plan.workspace.numel()
    say("workspace", size)
    assert size > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        keep_busy()
        plan.run()
    del plan
    junk = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert junk.data_ptr() != address
    assert same([y], [want])


def test_a_block_run_on_an_ambient_stream_and_dropped():
    import torch
    m = Mlp(300, 136, 520, 72, "bf16", "silu", "int8", seed=6)
    m.forward().backward()
    want = bits([m.mlp.y, m.mlp.d_x])
    block = m.mlp
    got = [block.y, block.d_x]
    for t in got:
        t.zero_()
    held = {t.data_ptr(): t.numel() for t in (block.workspace, block.d_a, block.d_b)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        keep_busy()
        m.forward().backward()
    m.mlp = block = None
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in held.values()]
    assert not held.keys() & {t.data_ptr() for t in junk}
    assert same(got, want)

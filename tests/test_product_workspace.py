"""The gated block's workspace for the tensors of a call, without a GPU: what is read
where it lies takes none of it, and a call asks for exactly what
muon_mlp_exact_workspace says."""

import ctypes

import pytest
import torch

from matrix_optimizer_step_muon_amd import layer, muon
from test_layer_streams import q8, world  # noqa: F401  (a fixture)
from test_product_abi import L, at, backward, forward, grads, last, mlp, no_gpu
from test_product_streams import on_cpu  # noqa: F401  (a fixture)

MIB = 1 << 20


def need(m, g=None):
    n = ctypes.c_size_t()
    assert L.muon_mlp_exact_workspace(m, g, ctypes.byref(n)) == 0, muon.last_error()
    return n.value


def worst(m):
    n = ctypes.c_size_t()
    assert L.muon_mlp_workspace(m, ctypes.byref(n)) == 0
    return n.value


def keep_nothing(m):
    m.a = m.b = m.s = muon.muon_q8()
    return m


SIZES = [(1, 8, 8, 8), (300, 200, 336, 136), (16, 33, 77, 19), (16, 640, 2048, 640), (1030, 1000, 2056, 520), (2048, 384, 4352, 384)]


@no_gpu
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,width,inner,out", SIZES)
def test_a_call_asks_for_exactly_this(rows, width, inner, out, dtype):
    e = 2 if dtype else 4
    for shift, ld in ((0, 0), (e, 0), (0, 3), (e, 8)):
        for keep in (True, False):
            for wanted in (True, False):
                m, g = mlp(rows, width, inner, out, dtype=dtype), grads(width, inner, out)
                m.x, m.ld_x, m.w_gate, m.w_down = m.x + shift, m.ld_x + ld, m.w_gate + shift, m.w_down + shift
                g.dy, g.ld_dy, g.d_a, g.ld_d_a = g.dy + shift, g.ld_dy + ld, g.d_a + shift, g.ld_d_a + ld
                if not wanted:
                    g.d_x = None
                    m.y = m.y if not keep else None
                fwd = m if keep else keep_nothing(mlp(rows, width, inner, out, dtype=dtype))
                if not keep:
                    fwd.x, fwd.ld_x, fwd.w_gate, fwd.w_down = m.x, m.ld_x, m.w_gate, m.w_down
                for d, call, n in ((fwd, lambda: forward(fwd), need(fwd)), (m, lambda: backward(m, g), need(m, g))):
                    assert n <= worst(d)
                    d.workspace_bytes = n
                    assert call() == -5, muon.last_error()      # up to the launch
                    if n:
                        d.workspace_bytes = n - 1
                        last(call(), -1, "are needed")
                    d.workspace_bytes = 1 << 31


def test_what_is_not_known_counts_as_unaligned():
    for dtype in (0, 1):
        m, g = mlp(300, 200, 336, 136, dtype=dtype), grads(200, 336, 136)
        full = max(need(m), need(m, g))
        m.x = m.w_gate = m.w_up = m.w_down = g.dy = g.d_a = g.d_b = None
        assert max(need(m), need(m, g)) == worst(m) and (full < worst(m)) == (dtype == 1)


def test_refusals_and_nothing_to_do():
    n = ctypes.c_size_t(7)
    m = mlp()
    assert L.muon_mlp_exact_workspace(None, None, ctypes.byref(n)) == -1 and L.muon_mlp_exact_workspace(m, None, None) == -1
    m.inner = 0
    last(L.muon_mlp_exact_workspace(m, grads(), ctypes.byref(n)), -1, "inner")
    assert need(mlp(rows=0)) == 0 and need(mlp(rows=0), grads()) == 0


def test_aligned_bf16_weights_are_not_copied():
    """Decoding: s, and pieces of sums. Training: s, dy (whose alignment is not known when
    the object is made) and pieces; the weights, 750 MiB, are nowhere."""
    m = keep_nothing(mlp(16, 5120, 25600, 5120))
    assert need(m) < 32 * MIB
    m = keep_nothing(mlp(1, 2048, 6144, 2048))
    assert need(m) == 2 * 6144 * 2                    # both by the kernels for few rows, s in two planes
    m, g = mlp(4096, 5120, 25600, 5120), grads(5120, 25600, 5120)
    s, dy, pieces = 4096 * 25600 * 2, 4096 * 5120 * 2, 256 * 1024 * 512
    assert s <= need(m) <= s + pieces
    g.dy = None
    assert dy <= need(m, g) <= dy + pieces
    g.dy, g.d_x = at(9), None
    assert need(m, g) <= pieces


def block(rows=64, width=256, inner=512, dtype=torch.bfloat16, **kw):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return layer.GatedMLP(z(rows, width), z(inner, width), z(inner, width), z(width, inner), **kw)


def test_the_objects_workspace(on_cpu):  # noqa: F811
    saved = lambda rows: tuple(q8(rows, 512) for _ in range(3))  # noqa: E731
    weights = 3 * 256 * 512 * 2
    few = block(rows=2, kind=None)
    assert few.workspace.numel() == few._c.workspace_bytes == 2 * 2 * 512 * 2
    m = block(saved=saved(64), need_d_x=False)
    n = block(saved=saved(64))
    for b in (m, n):
        s = 64 * 512 * 2
        pieces = max(need(b._c), need(b._c, b._grads)) - s
        assert s <= b.workspace.numel() and pieces < 2 * MIB
        b._grads.dy = b.y.data_ptr() + 2               # any dy will do
        b._grads.ld_dy = 257
        assert need(b._c, b._grads) <= b.workspace.numel()
    f32 = block(rows=64, dtype=torch.float32, saved=saved(64))
    assert f32.workspace.numel() > 3 * weights          # three planes of all operands

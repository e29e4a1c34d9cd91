"""The C ABI of the layers' products without a GPU: struct layouts, and arguments that
are refused before any HIP call (the device addresses are made up, and nothing is
dereferenced). A call that is refused for what the test plants is right up to that:
without the mistake it gets as far as the launch, which reports HIP where there is
no GPU."""

import ctypes
import math
import os
import subprocess

import pytest

from matrix_optimizer_step_muon_amd import layer, muon

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000
STEP = 1 << 32
L = muon.lib()


def gpu_visible():
    import torch
    return torch.cuda.is_available()


# Valid descriptors at made-up addresses must never reach a kernel.
no_gpu = pytest.mark.skipif(gpu_visible(), reason="made-up device addresses: CPU only")


def at(i):
    return BASE + i * STEP


def q8(i, rows=40, cols=100, kind=0):
    return muon.muon_q8(at(i), at(i) + STEP // 2, rows, cols, -(-cols // 16) * 16, -(-cols // 32), kind, 0)


def mlp(rows=40, width=64, inner=100, out=72, dtype=muon.MUON_BF16, kind=0):
    return muon.muon_mlp(rows, width, inner, out, at(0), width, at(1), at(2), at(3), at(4), out, q8(5, rows, inner, kind),
                         q8(6, rows, inner, kind), q8(7, rows, inner, kind), at(8), 1 << 31, 0, dtype)


def grads(width=64, inner=100, out=72):
    return muon.muon_mlp_grads(at(9), out, at(10), width, at(11), inner, at(12), inner)


def w8(i=13, n=72, k=100):
    return muon.muon_w8(at(i), at(i + 1), at(i + 2), n, k, -(-k // 16) * 16, -(-n // 16) * 16, -(-k // 128))


def item(i=0, rows=40, n=72, k=100, transposed=0):
    b = 20 * i
    x = q8(b, rows, n if transposed else k, 1)
    out = k if transposed else n
    return muon.muon_linear8_item(x, w8(b + 1, n, k), at(b + 4), out, at(b + 5), out, 1.0, transposed)


def last(status, code, message):
    assert status == code and message in muon.last_error(), (status, muon.last_error())


def forward(m):
    return L.muon_mlp_forward(m, None)


def backward(m, g):
    return L.muon_mlp_backward(m, g, None)


def product(it, n=1, dtype=1, ws=at(1000), nbytes=1 << 31):
    return L.muon_linear8(it, n, dtype, ws, nbytes, None)


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    names = ("muon_mlp", "muon_mlp_grads", "muon_w8", "muon_linear8_item")
    lines = []
    for n in names:
        for f, _ in getattr(muon, n)._fields_:
            lines.append(f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));')
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
    for act, code in layer.ACTS.items():
        lines.append(f'printf("act.{act} %d\\n", MUON_ACT_{act.upper()});')
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void) {' + "".join(lines) + "return 0;}")
    exe = tmp_path / "s"
    subprocess.run(["gcc", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for n in names:
        t = getattr(muon, n)
        assert int(got[n]) == ctypes.sizeof(t), n
        for f, _ in t._fields_:
            assert int(got[f"{n}.{f}"]) == getattr(t, f).offset, (n, f)
    for act, code in layer.ACTS.items():
        assert int(got[f"act.{act}"]) == code


def set_path(obj, path, value):
    *head, leaf = path.split(".")
    for h in head:
        obj = getattr(obj, h)
    setattr(obj, leaf, value)


@no_gpu
def test_valid_calls_reach_the_launch():
    none = muon.muon_q8()
    for m in (mlp(), mlp(dtype=0), mlp(rows=3), mlp(kind=1)):
        assert forward(m) == -5 and backward(m, grads()) == -5, muon.last_error()
        m.a = m.b = m.s = none
        assert forward(m) == -5, muon.last_error()
    m, g = mlp(), grads()
    m.y = None
    g.d_x = None
    assert forward(m) == -5 and backward(m, g) == -5, muon.last_error()
    m.x = m.s.q = None
    assert backward(m, g) == -5, muon.last_error()   # reads neither
    for t in (0, 1):
        assert product(item(transposed=t)) == -5 and product(item(transposed=t), dtype=0) == -5, muon.last_error()
        assert product(item(rows=2, transposed=t)) == -5, muon.last_error()
    assert L.muon_w8_save(at(40), 100, 1, w8(), None) == -5 and L.muon_w8_load(w8(), at(40), 100, 0, None) == -5
    w = w8()
    w.qt = None
    assert L.muon_w8_save(at(40), 100, 0, w, None) == -5, muon.last_error()


@no_gpu
def test_nothing_to_do_is_no_error():
    m = mlp(rows=0)
    m.x = m.y = m.workspace = None
    m.a.q = m.b.q = m.s.q = None
    assert forward(m) == 0, muon.last_error()
    it = item(rows=0)
    it.x.q = it.x.e = it.y = it.c = None
    assert product(it, ws=None, nbytes=0) == 0, muon.last_error()


@pytest.mark.parametrize("path,value,code,message", [
    ("rows", -1, -1, "rows must be"), ("rows", 1 << 31, -1, "rows must be"), ("width", 0, -1, "width must be"),
    ("inner", (1 << 22) + 1, -1, "inner must be"), ("out", 0, -1, "out must be"), ("dtype", 2, -4, "dtype"),
    ("act", 4, -4, "act"), ("act", -1, -4, "act"), ("x", None, -1, "x is NULL"), ("ld_x", 63, -1, "x: row stride"),
    ("x", at(0) + 1, -3, "x is not 2-byte"), ("w_gate", None, -1, "w_gate is NULL"), ("w_up", at(2) + 1, -3, "w_up is not 2-byte"),
    ("w_down", None, -1, "w_down is NULL"), ("ld_y", 71, -1, "y: row stride"), ("ld_y", (1 << 22) + 1, -1, "2^22"),
    ("a.cols", 99, -1, "a must be"), ("b.rows", 39, -1, "b must be"), ("s.kind", 2, -4, "kind"), ("s.kind", 1, -1, "same kind"),
    ("a.ldq", 113, -3, "multiple of 16"), ("b.e", None, -1, "b is NULL"), ("workspace", None, -1, "workspace is NULL"),
    ("workspace", at(8) + 8, -3, "workspace is not 16-byte"), ("workspace_bytes", 100, -1, "are needed"),
    ("y", at(0) + 64, -2, "overlaps"), ("a.q", at(6), -2, "overlaps"), ("y", at(8) + 64, -2, "overlaps"), ("y", at(3), -2, "overlaps"),
])
def test_forward_refusals(path, value, code, message):
    m = mlp()
    set_path(m, path, value)
    last(forward(m), code, message)


def test_forward_that_writes_nothing():
    m = mlp()
    m.y = m.a.q = m.b.q = m.s.q = None
    last(forward(m), -1, "are all NULL")
    assert L.muon_mlp_forward(None, None) == -1 and L.muon_mlp_backward(None, grads(), None) == -1
    assert L.muon_mlp_backward(mlp(), None, None) == -1


@pytest.mark.parametrize("what,path,value,code,message", [
    ("m", "a.q", None, -1, "a is NULL"), ("m", "b.cols", 101, -1, "b must be"), ("m", "b.kind", 1, -1, "same kind"),
    ("m", "workspace_bytes", 0, -1, "are needed"), ("m", "act", 9, -4, "act"), ("m", "dtype", 3, -4, "dtype"),
    ("g", "dy", None, -1, "dy is NULL"), ("g", "ld_dy", 71, -1, "dy: row stride"), ("g", "d_a", None, -1, "d_a is NULL"),
    ("g", "d_b", at(12) + 1, -3, "d_b is not 2-byte"), ("g", "ld_d_a", 99, -1, "d_a: row stride"),
    ("g", "ld_d_b", (1 << 22) + 1, -1, "2^22"), ("g", "ld_d_x", (1 << 22) + 1, -1, "2^22"), ("g", "ld_d_x", 63, -1, "d_x: row stride"),
    ("g", "d_a", at(12), -2, "overlaps"), ("g", "d_x", at(9), -2, "overlaps"), ("g", "d_b", at(5), -2, "overlaps"),
    ("g", "d_x", at(1), -2, "overlaps"), ("g", "d_a", at(8), -2, "overlaps"),
])
def test_backward_refusals(what, path, value, code, message):
    m, g = mlp(), grads()
    set_path(m if what == "m" else g, path, value)
    last(backward(m, g), code, message)


def test_block_workspace():
    n = ctypes.c_size_t()
    m = mlp()
    assert L.muon_mlp_workspace(m, ctypes.byref(n)) == 0 and n.value >= 40 * 104 * 2
    m.rows = 0
    assert L.muon_mlp_workspace(m, ctypes.byref(n)) == 0 and n.value == 0
    assert L.muon_mlp_workspace(m, None) == -1 and L.muon_mlp_workspace(None, ctypes.byref(n)) == -1
    m.width = 0
    last(L.muon_mlp_workspace(m, ctypes.byref(n)), -1, "width")


@no_gpu
def test_the_workspace_covers_every_alignment():
    """What muon_mlp_workspace says is enough for tensors at any address and stride, and
    the calls ask for no more."""
    n = ctypes.c_size_t()
    for dtype in (0, 1):
        for sizes in ((1, 8, 8, 8), (300, 200, 336, 136), (16, 33, 77, 19), (1030, 1000, 2056, 520), (2048, 384, 4352, 384)):
            m = mlp(*sizes, dtype=dtype)
            assert L.muon_mlp_workspace(m, ctypes.byref(n)) == 0
            e = 2 if dtype else 4
            for shift, ld in ((0, 0), (e, 0), (0, 3), (e, 8)):
                m = mlp(*sizes, dtype=dtype)
                g = grads(sizes[1], sizes[2], sizes[3])
                m.workspace_bytes = n.value
                m.x, m.ld_x, m.w_gate, m.w_down = m.x + shift, m.ld_x + ld, m.w_gate + shift, m.w_down + shift
                g.dy, g.ld_dy, g.d_a, g.ld_d_a = g.dy + shift, g.ld_dy + ld, g.d_a + shift, g.ld_d_a + ld
                assert forward(m) == -5 and backward(m, g) == -5, (sizes, shift, ld, muon.last_error())


@pytest.mark.parametrize("path,value,code,message", [
    ("q", None, -1, "weight is NULL"), ("e", None, -1, "weight is NULL"), ("n", 0, -1, "n and k"), ("k", (1 << 24) + 1, -1, "n and k"),
    ("ldq", 96, -1, "row stride"), ("ldq", 113, -3, "multiple of 16"), ("ldqt", 73, -3, "multiple of 16"), ("ldqt", 64, -1, "row stride"),
    ("q", at(13) + 8, -3, "16-byte"), ("lde", 0, -1, "row stride"), ("qt", at(13), -2, "overlaps"), ("e", at(14) + 16, -2, "overlaps"),
])
def test_weight_refusals(path, value, code, message):
    w = w8()
    set_path(w, path, value)
    last(L.muon_w8_save(at(40), 100, 1, w, None), code, message)
    if path not in ("qt", "ldqt") and code != -2:
        last(L.muon_w8_load(w, at(40), 100, 1, None), code, message)


@pytest.mark.parametrize("x,ldx,dtype,code,message", [
    (None, 100, 1, -1, "w is NULL"), (at(40), 99, 1, -1, "row stride"), (at(40) + 1, 100, 1, -3, "2-byte"),
    (at(40) + 2, 100, 0, -3, "4-byte"), (at(40), 100, 2, -4, "dtype"), (at(13) + 16, 100, 1, -2, "overlaps"),
])
def test_weight_tensor_refusals(x, ldx, dtype, code, message):
    last(L.muon_w8_save(x, ldx, dtype, w8(), None), code, message)
    last(L.muon_w8_load(w8(), x, ldx, dtype, None), code, message)
    assert L.muon_w8_save(at(40), 100, 1, None, None) == -1


@pytest.mark.parametrize("path,value,code,message", [
    ("x.kind", 0, -4, "e4m3"), ("x.cols", 99, -1, "columns"), ("x.q", None, -1, "x is NULL"), ("x.rows", -1, -1, "rows must be"),
    ("w.q", None, -1, "w is NULL"), ("w.e", None, -1, "w is NULL"), ("w.n", 0, -1, "n and k"), ("w.ldq", 40, -3, "multiple of 16"),
    ("y", None, -1, "y is NULL"), ("ld_y", 71, -1, "y: row stride"), ("ld_y", (1 << 22) + 1, -1, "2^22"), ("y", at(4) + 1, -3, "2-byte"),
    ("beta", math.nan, -1, "beta"), ("beta", math.inf, -1, "beta"), ("c", None, -1, "c is NULL"), ("ld_c", 71, -1, "c: row stride"),
    ("ld_c", (1 << 22) + 1, -1, "2^22"), ("c", at(4) + 4, -2, "overlaps"), ("y", at(0), -2, "overlaps"), ("y", at(1) + 64, -2, "overlaps"),
])
def test_product_refusals(path, value, code, message):
    it = item()
    set_path(it, path, value)
    last(product(it), code, "item 0: ")
    assert message in muon.last_error()
    n = ctypes.c_size_t()
    last(L.muon_linear8_workspace(it, 1, 1, ctypes.byref(n)), code, message)


def test_more_product_refusals():
    it = item(transposed=1)
    it.w.qt = None
    last(product(it), -1, "w.qt is NULL")
    it = item()
    it.c, it.ld_c = it.y, it.ld_y + 8
    last(product(it), -1, "another row stride")
    last(product(None), -1, "items is NULL")
    last(product(item(), n=0), -1, "n_items")
    last(product(item(), dtype=2), -4, "dtype")
    huge = item(rows=1 << 29, n=4096, k=64)
    huge.w = w8(-3, 4096, 64)
    huge.x.e, huge.y, huge.beta = BASE + (1 << 42), BASE + (1 << 44), 0.0
    last(product(huge), -1, "2^22 tiles")
    wide = item(n=(1 << 22) + 16, k=64)
    last(product(wide), -1, "2^22")
    two = (muon.muon_linear8_item * 2)(item(0), item(1))
    two[1].y = two[0].y
    last(L.muon_linear8(two, 2, 1, at(1000), 1 << 31, None), -2, "overlaps")
    long = item(rows=40, n=64, k=1 << 20)      # few tiles: in pieces
    n = ctypes.c_size_t()
    assert L.muon_linear8_workspace(long, 1, 1, ctypes.byref(n)) == 0 and n.value > 0
    last(product(long, nbytes=n.value - 1), -1, "are needed")
    last(product(long, ws=None), -1, "workspace is NULL")
    last(product(long, ws=at(1000) + 8), -3, "16-byte")
    last(product(long, ws=at(4), nbytes=1 << 31), -2, "overlaps")
    assert L.muon_linear8_workspace(item(), 1, 1, None) == -1


def test_python_refuses_what_it_can_see():
    import torch
    cpu = torch.zeros(4, 8)
    for f in (lambda: layer.GatedMLP(cpu, cpu, cpu, cpu), lambda: layer.GatedMLP(cpu, cpu, cpu, cpu, act="swish"),
              lambda: layer.Linear8([]), lambda: layer.Linear8([(cpu, cpu, cpu)])):
        with pytest.raises(layer.MuonError):
            f()
    with pytest.raises(layer.MuonError):
        layer.W8(0, 4)

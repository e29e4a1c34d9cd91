"""The layer operators' C ABI without a GPU: struct layouts, and arguments that
are refused before any HIP call (the device addresses are made up, and nothing
is dereferenced). A call that is refused for what the test plants is right up
to that: without the mistake it gets as far as the launch, which reports HIP
where there is no GPU."""

import copy
import ctypes
import math
import os
import subprocess

import pytest

from matrix_optimizer_step_muon_amd import layer, muon

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000
STEP = 1 << 28
L = muon.lib()


def gpu_visible():
    import torch
    return torch.cuda.is_available()


# Valid descriptors at made-up addresses must never reach a kernel.
no_gpu = pytest.mark.skipif(gpu_visible(), reason="made-up device addresses: CPU only")


def at(i):
    return BASE + i * STEP


def q8(i, rows=40, cols=100, kind=0):
    return muon.muon_q8(at(i), at(i) + STEP // 2, rows, cols, 112, 4, kind, 0)


def site(rows=40, cols=100, dtype=muon.MUON_BF16):
    return muon.muon_norm_site(rows, cols, at(0), cols, at(1), cols, at(2), at(3), at(4), 0, at(5), cols, at(6), cols,
                               at(7), at(8), q8(9, rows, cols), q8(10, rows, cols), 1.0, 1.0, 1e-6, dtype)


def grads(cols=100):
    return muon.muon_norm_grads(at(11), cols, at(12), cols, at(13), cols, at(14), cols, at(15), at(16), at(17), 0, at(18), 1 << 24)


def item(i=0, rows=40, n=64, k=100):
    b = 20 * i
    return muon.muon_wgrad_item(at(b), n, q8(b + 1, rows, k), at(b + 2), at(b + 3), at(b + 4), n, 1.0, 0)


def last(status, code, message):
    assert status == code and message in muon.last_error(), (status, muon.last_error())


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    names = ("muon_q8", "muon_norm_site", "muon_norm_grads", "muon_wgrad_item")
    lines = []
    for n in names:
        for f, _ in getattr(muon, n)._fields_:
            lines.append(f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));')
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void) {' + "".join(lines) + "return 0;}")
    exe = tmp_path / "s"
    subprocess.run(["gcc", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for n in names:
        t = getattr(muon, n)
        assert int(got[n]) == ctypes.sizeof(t), n
        for f, _ in t._fields_:
            assert int(got[f"{n}.{f}"]) == getattr(t, f).offset, (n, f)


def set_path(obj, path, value):
    *head, leaf = path.split(".")
    for h in head:
        obj = getattr(obj, h)
    setattr(obj, leaf, value)


@no_gpu
def test_valid_calls_reach_the_launch():
    s, g, p = site(), grads(), q8(0)
    for st in (L.muon_q8_save(at(5), 100, 1, p, None), L.muon_q8_load(p, at(5), 100, 0, None), L.muon_norm_forward(s, None),
               L.muon_norm_backward(s, g, None), L.muon_wgrad(item(), 1, 1, 0, at(30), 1 << 30, None)):
        assert st == -5, muon.last_error()


@pytest.mark.parametrize("save", [True, False])
@pytest.mark.parametrize("path,value,code,message", [
    ("q", None, -1, "checkpoint is NULL"), ("e", None, -1, "checkpoint is NULL"), ("q", at(0) + 8, -3, "16-byte"),
    ("rows", -1, -1, "rows must be"), ("rows", 1 << 31, -1, "rows must be"), ("cols", 0, -1, "cols must be"),
    ("cols", (1 << 24) + 1, -1, "cols must be"), ("ldq", 96, -1, "row stride"), ("ldq", 113, -3, "multiple of 16"),
    ("lde", 3, -1, "row stride"), ("kind", 2, -4, "kind"), ("kind", -1, -4, "kind"), ("ldq", 1 << 25, -1, "row stride"),
    ("e", at(0) + 64, -2, "overlaps"),
])
def test_checkpoint_refusals(save, path, value, code, message):
    p = q8(0)
    set_path(p, path, value)
    if code == -2 and not save:
        pytest.skip("read-only views may overlap")
    last(L.muon_q8_save(at(5), 100, 1, p, None) if save else L.muon_q8_load(p, at(5), 100, 1, None), code, message)


@pytest.mark.parametrize("x,ldx,dtype,code,message", [
    (None, 100, 1, -1, "x is NULL"), (at(5), 99, 1, -1, "row stride"), (at(5) + 1, 100, 1, -3, "2-byte"),
    (at(5) + 2, 100, 0, -3, "4-byte"), (at(5), 100, 2, -4, "dtype"), (at(0) + 16, 100, 1, -2, "overlaps"),
    (at(0) + STEP // 2 - 2, 100, 1, -2, "overlaps"),
])
def test_checkpoint_tensor_refusals(x, ldx, dtype, code, message):
    last(L.muon_q8_save(x, ldx, dtype, q8(0), None), code, message)
    last(L.muon_q8_load(q8(0), x, ldx, dtype, None), code, message)


def test_null_descriptors():
    n = ctypes.c_size_t()
    assert L.muon_q8_save(at(5), 100, 1, None, None) == -1
    assert L.muon_q8_load(None, at(5), 100, 1, None) == -1
    assert L.muon_norm_forward(None, None) == -1
    assert L.muon_norm_backward(None, grads(), None) == -1 and L.muon_norm_backward(site(), None, None) == -1
    assert L.muon_wgrad(None, 1, 1, 1, None, 0, None) == -1
    assert L.muon_wgrad_workspace(item(), 1, 1, 1, None) == -1
    assert L.muon_norm_backward_workspace(4, 4, None) == -1
    assert L.muon_norm_backward_workspace(4, 32769, ctypes.byref(n)) == -4
    assert L.muon_norm_backward_workspace(-1, 4, ctypes.byref(n)) == -1


@pytest.mark.parametrize("path,value,code,message", [
    ("rows", -2, -1, "rows must be"), ("cols", 0, -1, "cols must be"), ("cols", 32769, -4, "32768"), ("dtype", 2, -4, "dtype"),
    ("eps", -1.0, -1, "eps must be"), ("eps", math.nan, -1, "finite"), ("res_scale", math.inf, -1, "finite"),
    ("branch_scale", math.nan, -1, "finite"), ("branch", None, -1, "branch is NULL"), ("residual", None, -1, "residual is NULL"),
    ("w_pre", None, -1, "w_pre is NULL"), ("y", None, -1, "y is NULL"), ("h", None, -1, "h is NULL"),
    ("ld_branch", 99, -1, "row stride"), ("ld_y", 0, -1, "row stride"), ("ld_gate", 50, -1, "row stride"),
    ("y", at(5) + 1, -3, "aligned"), ("rstd_y", at(7) + 2, -3, "aligned"), ("u.ldq", 100, -3, "multiple of 16"),
    ("u.rows", 39, -1, "rows x cols"), ("v.cols", 99, -1, "rows x cols"), ("v.kind", 5, -4, "kind"), ("u.e", None, -1, "u is NULL"),
    ("y", at(0), -2, "overlaps"), ("h", at(5) + 2, -2, "overlaps"), ("y", at(2), -2, "overlaps"), ("h", at(9), -2, "overlaps"),
    ("rstd_y", at(8) + 8, -2, "overlaps"),
])
def test_norm_forward_refusals(path, value, code, message):
    s = site()
    set_path(s, path, value)
    last(L.muon_norm_forward(s, None), code, message)


@pytest.mark.parametrize("path,value,code,message", [
    ("g.dh", None, -1, "dh is NULL"), ("g.ld_dh", 99, -1, "row stride"), ("g.d_residual", None, -1, "d_residual is NULL"),
    ("g.d_branch", None, -1, "d_branch is NULL"), ("s.rstd_y", None, -1, "rstd_y is NULL"), ("s.rstd_b", None, -1, "rstd_b is NULL"),
    ("s.u.q", None, -1, "u is NULL"), ("s.v.q", None, -1, "v is NULL"), ("s.w_post", None, -1, "no w_post"),
    ("s.gate", None, -1, "no gate"), ("g.workspace_bytes", 1000, -1, "workspace has 1000"), ("g.workspace", None, -1, "workspace is NULL"),
    ("g.workspace", at(18) + 8, -3, "workspace"), ("g.d_w_pre", at(15) + 1, -3, "aligned"), ("g.d_branch", at(12), -2, "overlaps"),
    ("g.d_residual", at(11), -2, "overlaps"), ("g.d_gate", at(16) + 20, -2, "overlaps"), ("g.workspace", at(13) - 64, -2, "overlaps"),
    ("g.d_residual", at(9) + 32, -2, "overlaps"),
])
def test_norm_backward_refusals(path, value, code, message):
    o = {"s": site(), "g": grads()}
    which, rest = path.split(".", 1)
    set_path(o[which], rest, value)
    last(L.muon_norm_backward(o["s"], o["g"], None), code, message)


@pytest.mark.parametrize("path,value,code,message", [
    ("dy", None, -1, "dy is NULL"), ("ld_dy", 63, -1, "row stride"), ("dy", at(20) + 1, -3, "aligned"), ("n", 0, -1, "n must be"),
    ("n", (1 << 24) + 1, -1, "n must be"), ("x.q", None, -1, "x is NULL"), ("x.rows", -1, -1, "rows must be"),
    ("x.cols", 0, -1, "cols must be"), ("x.kind", 1, -1, "same kind"), ("g", None, -1, "g is NULL"), ("g", at(23) + 8, -3, "16-byte"),
    ("c", None, -1, "c is NULL"), ("c", at(24) + 4, -3, "16-byte"), ("scale", at(22) + 1, -3, "aligned"),
    ("beta", math.nan, -1, "beta"), ("beta", math.inf, -1, "beta"), ("g", at(20) + 16, -2, "item 1: "), ("g", at(3) + 64, -2, "overlaps"),
    ("c", at(23) + 64, -2, "overlaps"), ("c", at(3), -2, "overlaps"), ("g", at(21) + 32, -2, "overlaps"),
])
def test_wgrad_refusals(path, value, code, message):
    items = (muon.muon_wgrad_item * 2)(item(0), item(1))
    set_path(items[1], path, value)
    last(L.muon_wgrad(items, 2, 1, 0, at(30), 1 << 24, None), code, message)


def test_wgrad_types_counts_and_workspace():
    one = (muon.muon_wgrad_item * 1)(item(0, rows=5000, n=300))
    last(L.muon_wgrad(one, 0, 1, 1, None, 0, None), -1, "n_items")
    last(L.muon_wgrad(one, 1, 2, 1, None, 0, None), -4, "dtype")
    last(L.muon_wgrad(one, 1, 1, 2, None, 0, None), -4, "g_dtype")
    need = ctypes.c_size_t()
    assert L.muon_wgrad_workspace(one, 1, 1, 0, ctypes.byref(need)) == 0 and need.value > 0
    last(L.muon_wgrad(one, 1, 1, 0, at(30), need.value - 1, None), -1, "workspace has")
    last(L.muon_wgrad(one, 1, 1, 0, None, need.value, None), -1, "workspace is NULL")
    last(L.muon_wgrad(one, 1, 1, 0, at(30) + 8, need.value, None), -3, "workspace")
    last(L.muon_wgrad(one, 1, 1, 0, at(3) + 64, need.value, None), -2, "workspace")
    # A large product of fp32 dY rewrites it as three bf16 planes of a width that is a multiple of 8.
    big = (muon.muon_wgrad_item * 1)(item(0, rows=5000, n=8100, k=6000))
    big[0].x.ldq, big[0].x.lde = 6000, 188
    assert L.muon_wgrad_workspace(big, 1, 0, 0, ctypes.byref(need)) == 0 and need.value >= 3 * 2 * 5000 * 8104


@no_gpu
def test_column_blocks_of_one_buffer_are_disjoint_and_c_may_be_g():
    s = site()
    s.y, s.ld_y, s.h, s.ld_h = at(5), 200, at(5) + 200, 200     # two column blocks of a 200-wide bf16 matrix
    assert L.muon_norm_forward(s, None) == -5
    s.h = at(5) + 198
    last(L.muon_norm_forward(s, None), -2, "overlaps")
    it = item()
    it.c = it.g
    assert L.muon_wgrad(it, 1, 1, 0, at(30), 1 << 24, None) == -5


@no_gpu
def test_views_without_rows_may_be_null():
    p = q8(0, rows=0)
    p.q = p.e = None
    assert L.muon_q8_save(None, 100, 1, p, None) == 0
    assert L.muon_q8_load(p, None, 100, 1, None) == 0


def test_python_refusals():
    import torch
    t = torch.zeros(4, 8)
    for call in (lambda: layer.NormSite(t, t, t[0]), lambda: layer._matrix(t, "x"),
                 lambda: layer.WGrad([]), lambda: layer.WGrad([(t, "x", t)]), lambda: layer.Q8(-1, 4), lambda: layer.Q8(1, 4, "int4"),
                 lambda: layer.Q8(1, 4, q=t)):
        with pytest.raises(muon.MuonError):
            call()

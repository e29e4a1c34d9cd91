"""Infinities in the gated block: what the definition says of them, NaN where it says
NaN, in bf16 and in fp32, whose products are sums of products of parts. The numbers
beside them include those that one part alone holds (bf16 numbers and powers of two)."""

import numpy as np
import pytest

from layer_helpers import dev, f64, say, stored, tdt
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref, product_ref as ref
from product_helpers import Mlp

pytestmark = pytest.mark.gpu

# what the operands beside the infinities hold: all 24 bits, the 8 of one part, or 1
NUMBERS = {"fp32": lambda a: a, "bf16": lambda a: stored(a, "bf16"),
           "powers": lambda a: np.sign(a) * 2.0 ** np.round(np.log2(np.abs(a) + 1e-3))}


def sync():
    import torch
    torch.cuda.synchronize()


def same_kind(got, want, what):
    """NaN, infinity by sign, or a number, as the definition has it."""
    for name, f in (("NaN", np.isnan), ("inf", np.isposinf), ("-inf", np.isneginf)):
        bad = f(got) != f(want)
        assert not bad.any(), (what, name, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def block(rows, inner, dtype, act, kind, numbers, edit):
    def change(m):
        for t in (m.x, m.wg, m.wu, m.wd, m.dy):
            t[:] = NUMBERS[numbers](t)
        edit(m)
    return Mlp(rows, 40, inner, 24, dtype, act, kind, seed=rows + inner, edit=change)


@pytest.mark.parametrize("numbers", list(NUMBERS))
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("rows,inner,kind", [(4, 56, None), (4, 56, "int8"), (40, 72, None), (150, 136, "e4m3"), (3, 1, None)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(dtype, rows, inner, kind, act, numbers):
    """Rows 1 and 2: an infinity that makes both sums of every inner column positive
    infinities, and y's sign that of its weights. Row 0 has one that meets zeros."""
    def edit(m):
        m.wg[:, 5], m.wu[:, 5] = np.abs(m.wg[:, 5]) + 0.5, np.abs(m.wu[:, 5]) + 0.5
        m.wg[:, 6], m.wu[:, 6] = -m.wg[:, 5], -m.wu[:, 5]
        m.wg[0, 7] = 0
        m.wd[:] = (np.abs(m.wd) + 0.125) * np.where(np.arange(24) % 2, -1, 1)[:, None]
        for t in (m.wg, m.wu, m.wd):
            t[:] = stored(t, dtype)
        m.x[1, 5], m.x[2, 6], m.x[0, 7] = np.inf, -np.inf, np.inf
    m = block(rows, inner, dtype, act, kind, numbers, edit)
    say(rows, inner, dtype, act, kind, numbers)
    m.forward()
    sync()
    with np.errstate(invalid="ignore"):
        y = ref.mlp_forward(m.x, m.wg, m.wu, m.wd, act)[3]
    assert np.isinf(y[1:3]).all() and np.isnan(y[0]).all()
    same_kind(f64(m.mlp.y), y, "y")
    if kind:
        for q in (m.mlp.a, m.mlp.b, m.mlp.s):
            e = q.e.cpu().numpy()
            assert (e[1:3] == 255).all() and not (e[3:] == 255).any()


@pytest.mark.parametrize("numbers", list(NUMBERS))
@pytest.mark.parametrize("rows,inner", [(4, 56), (40, 72), (150, 136), (3, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(dtype, rows, inner, numbers):
    def edit(m):
        m.wg[:], m.wu[:] = np.abs(m.wg) + 0.125, np.abs(m.wu) + 0.125
        m.wd[:] = np.abs(m.wd) + 0.125
        m.x[:] = np.abs(m.x) + 0.125             # a, b and act'(a) above 0
        for t in (m.x, m.wg, m.wu, m.wd):
            t[:] = stored(t, dtype)
        m.dy[1, 3], m.dy[2, 9] = np.inf, -np.inf
    m = block(rows, inner, dtype, "silu", "int8", numbers, edit)
    say(rows, inner, dtype, numbers)
    m.forward().backward()
    sync()
    from layer_helpers import codes
    a, b = (layer_ref.q8_decode(*codes(q), "int8") for q in (m.mlp.a, m.mlp.b))
    with np.errstate(invalid="ignore"):
        _, da, db, dx = ref.mlp_backward(m.dy, a, b, m.wg, m.wu, m.wd, "silu")
    assert np.isposinf(dx[1]).all() and np.isneginf(dx[2]).all()
    for name, want in (("d_a", da), ("d_b", db), ("d_x", dx)):
        same_kind(f64(getattr(m.mlp, name)), want, name)


@pytest.mark.parametrize("rows,kind", [(4, None), (40, "int8")])
def test_a_product_that_overflows_is_an_infinity(rows, kind):
    """act(a) b past the largest number: s is an infinity, y one of its weights' sign,
    for weights of one bit as for others."""
    import torch
    w = torch.ones(1, 8, device="cuda")
    down = dev(np.array([[1.0], [-2.0], [0.3], [-1.7]]), "f32")
    x = torch.full((rows, 8), 1e24, device="cuda")
    m = layer.GatedMLP(x, w, w.clone(), down, act="relu", kind=kind)
    m.forward()
    sync()
    same_kind(f64(m.y), np.repeat([[np.inf, -np.inf, np.inf, -np.inf]], rows, 0), "y")


def test_zeros_stay_zeros():
    """Zeros have no sign to keep: their products are zeros, and NaNs with an infinity."""
    import torch
    for rows, kind in ((4, None), (40, "int8")):
        x, w = torch.zeros(rows, 40, device="cuda"), torch.randn(56, 40, device="cuda")
        m = layer.GatedMLP(x, w, w.clone(), torch.randn(24, 56, device="cuda"), act="relu", kind=kind)
        m.forward()
        sync()
        assert bool((m.y == 0).all()) and m.y.dtype == tdt("f32")
        x[0, 3] = float("inf")
        w[:, 3] = 0
        m.forward()
        sync()
        assert bool(torch.isnan(m.y[0]).all()) and bool((m.y[1:] == 0).all())

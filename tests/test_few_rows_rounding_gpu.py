"""Decoding one token or two in bf16 rounds once: between the two kernels for few rows s
keeps 16 bits, so y is the bf16 number next to the exact one, but where that lies by a
border.

How often it may not be: s is off by 2^-16 at most, 2^-17 in the mean, and so is y against
its typical size; a border lies within an error d of a number with the probability 2 d /
(a step of 2^-8 to 2^-7 of it), 2^-9 for numbers of typical size, a few times that for the
small ones among them: 5% allows for ten times. With s in bf16, 2^-9 off in the mean, it
would be every other number."""

import numpy as np
import pytest

from layer_helpers import f64, say, stored
from matrix_optimizer_step_muon_amd import layer
from oracle import product_ref as ref
from product_helpers import Mlp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("width,inner,out", [(2048, 640, 520), (129, 1000, 1033), (640, 4100, 1000), (200, 300, 4500), (64, 131, 8200)])
def test_one_rounding(width, inner, out, rows, act):
    import torch
    m = Mlp(rows, width, inner, out, "bf16", act, None, seed=rows + out)
    cut = [c["tile"] for c in m.mlp.info()["forward"]]
    m.forward()
    torch.cuda.synchronize()
    m.check_forward()
    assert cut == [0, 0]
    want = ref.mlp_forward(m.x, m.wg, m.wu, m.wd, act)[3]
    other = float(np.mean(f64(m.mlp.y) != stored(want, "bf16")))
    say(width, inner, out, rows, act, f"{100 * other:.2f}%")
    assert other < 0.05


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("inner", [56, 131])
def test_infinities_meet_both_planes(rows, inner):
    """An infinite s, and infinite weights against s that the first plane holds alone."""
    import torch
    one = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    down = one(24, inner)
    down[1::2] = -1
    x = one(rows, 8)
    x[-1] = 2
    for act, gate in (("relu", one(inner, 8)), ("silu", one(inner, 8))):
        m = layer.GatedMLP(x.clone(), gate, gate.clone(), down, act=act, kind=None)
        assert [c["tile"] for c in m.info()["forward"]] == [0, 0]
        down[3, 5], down[4, inner - 1] = float("inf"), -float("inf")
        m.workspace.fill_(255)                        # nothing of it is read before it is written
        m.forward()
        torch.cuda.synchronize()
        assert bool((m.y[:, 3] == float("inf")).all()) and bool((m.y[:, 4] == -float("inf")).all())
        rest = [c for c in range(24) if c not in (3, 4)]
        assert bool(torch.isfinite(m.y[:, rest]).all())
        down[3, 5], down[4, inner - 1] = -1, 1
        m.x[0, 2] = float("inf")
        m.forward()
        torch.cuda.synchronize()
        assert bool((m.y[0, 0::2] == float("inf")).all()) and bool((m.y[0, 1::2] == -float("inf")).all())
        assert bool(torch.isfinite(m.y[1:]).all())


def test_the_same_bits_whatever_the_workspace_held():
    import torch
    for rows in (1, 2):
        m = Mlp(rows, 201, 331, 77, "bf16", "gelu", None, seed=rows)
        m.forward()
        torch.cuda.synchronize()
        want = m.mlp.y.clone()
        for byte in (0, 255, 0x7F):
            m.mlp.workspace.fill_(byte)
            m.forward()
            torch.cuda.synchronize()
            assert torch.equal(m.mlp.y, want)

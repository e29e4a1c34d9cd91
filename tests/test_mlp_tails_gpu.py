"""act(a) and act'(a) element by element where they are small: far left of 0, against
fp64. d_b = ds act(a) and d_a = ds b act'(a) show them, with ds = b = 1.

Bounds, in relative units of 2^-24. A constant is off by 1/2, an operation by 1, the
hardware's exponential, reciprocal and erfc by 2, 2 and 4 (twice their unit).
  silu       e^-a: its argument (constant, product) 1.5 |a|; then 2 + 2 and up to three
             operations: 1.5 |a| + 8
  gelu       erfc at |a| c: 1.5 of the argument, times the logarithm's slope, at most
             2 z^2 + 1 = a^2 + 1: 1.5 a^2 + 8 for Phi and a Phi. The density's
             argument a^2 / 2 has a constant and two products: 1.25 a^2 + 6
  gelu_tanh  the argument u = 1.596 a (1 + 0.0447 a^2): two constants and four operations,
             6 |u| with the exponential's own product; + 10
A derivative is a sum of two such terms; each counts by its size, plus two operations.
For bf16 a rounding more."""

import math

import numpy as np
import pytest

from layer_helpers import F32, HALF, dev, device_q8, f64, tdt, within
from matrix_optimizer_step_muon_amd import layer
from oracle import product_ref as ref

pytestmark = pytest.mark.gpu


def both(a, act):
    """act(a), act'(a), and what they may be off by. The tanh form is written with e^-u,
    since 1 + tanh is 0 or noise far left of 0 in 64 bits too."""
    f, df = ref.activation(a, act)
    if act == "relu":
        return f, df, 0 * a, 0 * a
    if act == "silu":
        s = 1 / (1 + np.exp(-a))
        rel = (1.5 * np.abs(a) + 8) * F32
        # 1 - s is off by what s is, and what is added to it is s
        return f, df, rel * np.abs(f), (rel + 4 * F32) * (s + np.abs(f))
    if act == "gelu":
        phi = 0.5 * np.vectorize(math.erfc)(-a / math.sqrt(2))
        pdf = np.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        rel = (1.5 * a * a + 8) * F32
        return f, df, rel * np.abs(f), (rel + 2 * F32) * (phi + np.abs(a) * pdf)
    u = 2 * math.sqrt(2 / math.pi) * a * (1 + 0.044715 * a * a)
    s, slope = 1 / (1 + np.exp(-u)), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * a * a)
    f, rel = a * s, (6 * np.abs(u) + 10) * F32
    return f, s + f * slope / (1 + np.exp(u)), rel * np.abs(f), (rel + 6 * F32) * (s + np.abs(f) * slope)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 70])
def test_activations_far_from_zero(rows, dtype, act):
    import torch
    # a in steps of 1/8 from -12 to 12: gelu_tanh's e^-u is a number down to -9.5
    low = -9 if act == "gelu_tanh" else -12
    q = np.repeat(np.arange(8 * low, 97)[None], rows, 0)
    inner = q.shape[1]
    one = np.full_like(q, 64)
    save = lambda c, e: device_q8(c.astype(np.int8).view(np.uint8), np.full((rows, -(-inner // 32)), 127 + e, np.uint8), "int8")  # noqa: E731
    dy, wd = np.zeros((rows, 8)), np.zeros((8, inner))
    dy[:, 0], wd[0] = 1, 1
    w = torch.zeros(inner, 16, dtype=tdt(dtype), device="cuda")
    m = layer.GatedMLP(torch.zeros(rows, 16, dtype=tdt(dtype), device="cuda"), w, w.clone(), dev(wd, dtype), act=act,
                       saved=(save(q, -3), save(one, -6)), need_d_x=False)
    m.backward(dev(dy, dtype))
    torch.cuda.synchronize()
    a = q / 8.0
    f, df, ef, edf = both(a, act)
    within(f64(m.d_b), f, ef + HALF[dtype] * (np.abs(f) + ef), "act")
    within(f64(m.d_a), df, edf + HALF[dtype] * (np.abs(df) + edf), "act'")

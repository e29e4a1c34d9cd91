"""Weight gradients of checkpoints at both ends of the exponent's range, against
the fp64 oracle. Every value a checkpoint stands for here is a finite fp32
number, and dY is scaled so that the gradient is one too.

Tolerances as in test_wgrad_gpu.py: one rounding to the gradient's type, and at
most one per product, two where the matrix instruction truncates."""

import numpy as np
import pytest

from layer_helpers import F32, HALF, dev, device_q8, f64, rng, say, stored, tdt, within
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu

# Each of the three kernels (tiles of 64, 128 and 256), with short last stages,
# odd and even numbers of stages, and the sum in pieces.
SIZES = [(40, 48, 64), (257, 40, 96), (300, 2048, 2048), (1000, 1024, 1100), (200, 4096, 4096), (330, 4096, 4100)]


def checkpoint(rows, cols, kind, exps, seed):
    g = rng(seed)
    e = g.choice(np.array(exps, np.uint8), (rows, -(-cols // 32)))
    # codes whose values stay below 2^128
    room = 2.0 ** (128 - (np.repeat(e, 32, 1)[:, :cols].astype(float) - 127))
    if kind == "int8":
        q = g.integers(-127, 128, (rows, cols))
        return np.where(np.abs(q) < room, q, q // 8).astype(np.int8).view(np.uint8), e
    q = g.integers(0, 127, (rows, cols)).astype(np.uint8)
    q = np.where(ref.e4m3_table()[q] < room, q, q & 0x3F).astype(np.uint8)
    return q | (g.integers(0, 2, (rows, cols)) * 128).astype(np.uint8), e


@pytest.mark.parametrize("kind,exps,power", [
    ("int8", (244, 245, 246, 247, 248, 249), -60), ("int8", (120, 245), -60), ("int8", (17, 18, 19), 20),
    ("e4m3", (244, 245, 246, 247), -60), ("e4m3", (17, 18, 19), 20)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_ends_of_the_exponents_range(rows, n, k, dtype, kind, exps, power):
    import torch
    say("case", rows, n, k, dtype, kind, exps)
    q, e = checkpoint(rows, k, kind, exps, rows + k)
    x = ref.q8_decode(q, e, kind)
    assert np.abs(x).max() < 2.0 ** 128
    dy = stored(rng(rows).standard_normal((rows, n)) * 2.0 ** power, dtype)
    G = torch.full((n, k), 9.0, dtype=tdt("f32"), device="cuda")
    layer.WGrad([(dev(dy, dtype), device_q8(q, e, kind), G)]).run()
    torch.cuda.synchronize()
    want, mag = ref.wgrad(dy, x), ref.wgrad(np.abs(dy), np.abs(x))
    within(f64(G), want, HALF["f32"] * np.abs(want) + (2 * rows + 40) * F32 * mag, "G")


@pytest.mark.parametrize("E,code,value", [(249, 0, 0.0), (249, 1, 2.0 ** 122), (254, 0, 0.0), (254, 0xFF, -2.0 ** 127),
                                          (249, 64, np.inf), (254, 2, np.inf), (255, 0, np.nan)])
@pytest.mark.parametrize("rows,n,k", [(40, 48, 64), (300, 2048, 2048), (200, 4096, 4096)])
def test_a_product_reads_the_values_that_loading_gives(rows, n, k, E, code, value):
    import torch
    say("case", rows, n, k, E, code)
    ckpt = device_q8(np.full((rows, k), code, np.uint8), np.full((rows, -(-k // 32)), E, np.uint8), "int8")
    x = torch.empty(rows, k, device="cuda")
    layer.q8_load(ckpt, x)
    G = torch.full((n, k), 9.0, device="cuda")
    layer.WGrad([(torch.full((rows, n), 2.0 ** -60, dtype=torch.bfloat16, device="cuda"), ckpt, G)]).run()
    torch.cuda.synchronize()
    assert np.array_equal(f64(x), np.full((rows, k), value), equal_nan=True)
    # every partial sum is a whole number of units below 2^24 of them: exact
    assert np.array_equal(f64(G), np.full((n, k), rows * 2.0 ** -60 * value), equal_nan=True)

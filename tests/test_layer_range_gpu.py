"""The ends of the number range, as the header states them: the largest values of
a checkpoint, and the smallest fp32 gradients that enter a weight gradient."""

import numpy as np
import pytest

from layer_helpers import codes, dev, device_q8, f64, rng, say, stored
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,top", [("int8", 1.984375), ("e4m3", 1.9375)])
def test_the_largest_values_of_a_checkpoint(kind, top, dtype):
    import torch
    big = 2.0 ** 127
    just = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    # int8 needs a top above the border, and rounds the border itself up then
    rows = [[top - just, 1.0], [top, 1.0], [top, -top - just], [-top - just, 1.0], [2 - just, 1.875], [1.75, 1.0]]
    x = np.zeros((len(rows), 40))
    x[:, [3, 9]] = np.array(rows) * big
    x = stored(x, dtype)
    ckpt = layer.q8_save(dev(x, dtype), layer.Q8(*x.shape, kind))
    outs = [torch.empty(*x.shape, device="cuda"), torch.empty(*x.shape, dtype=torch.bfloat16, device="cuda")]
    for o in outs:
        layer.q8_load(ckpt, o)
    torch.cuda.synchronize()
    wq, we = ref.q8_encode(x, kind)
    q, e = codes(ckpt)
    assert np.array_equal(q, wq) and np.array_equal(e, we)
    want = ref.q8_decode(wq, we, kind)
    over = np.abs(want) >= 2.0 ** 128
    for o in outs:
        assert np.array_equal(f64(o), np.where(over, np.copysign(np.inf, want), want))
    border = np.abs(x) >= top * big
    if kind == "int8":
        border &= np.abs(x).max(1, keepdims=True) > top * big
    assert np.array_equal(over, border)


@pytest.mark.parametrize("rows,n,k", [(40, 48, 64), (260, 2560, 2500), (200, 4096, 4096)])
@pytest.mark.parametrize("power", [-110, -120, -128, -140])
def test_small_fp32_gradients_lose_what_lies_below_the_smallest_bf16_number(rows, n, k, power):
    import torch
    say("case", rows, n, k, power)
    dy = np.zeros((rows, n))
    dy[rows // 3] = stored(rng(rows).uniform(1, 2, n) * 2.0 ** power, "f32")   # one token each: no sum to round
    q = rng(1).integers(-127, 128, (rows, k)).astype(np.int8)
    G = torch.empty(n, k, device="cuda")
    layer.WGrad([(dev(dy, "f32"), device_q8(q.view(np.uint8), np.full((rows, -(-k // 32)), 127 + 60, np.uint8), "int8"), G)]).run()
    torch.cuda.synchronize()
    x = q[rows // 3].astype(float) * 2.0 ** 60
    want = np.outer(dy[rows // 3], x)
    lost = 2.0 ** -133 if power < -110 else 0.0
    # three products of at most 16 bits, added with one rounding each
    tol = 4 * 2.0 ** -23 * np.abs(want) + lost * np.abs(x)
    assert (np.abs(f64(G) - want) <= tol).all()


@pytest.mark.parametrize("rows,n,k", [(40, 48, 64), (300, 2048, 2048), (200, 4096, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,E,code", [("int8", 249, 64), ("e4m3", 247, 0x78)])
def test_an_infinite_value_shows_in_its_column_only(rows, n, k, dtype, kind, E, code):
    import torch
    say("case", rows, n, k, dtype, kind)
    q, e = np.ones((rows, k), np.uint8), np.full((rows, -(-k // 32)), 127, np.uint8)
    q[rows // 2, 40], e[rows // 2, 1] = code, E
    dy = np.ones((rows, n)) * 2.0 ** -60
    G = torch.empty(n, k, device="cuda")
    layer.WGrad([(dev(dy, dtype), device_q8(q, e, kind), G)]).run()
    torch.cuda.synchronize()
    got = f64(G)
    assert not np.isfinite(got[:, 40]).any()
    got[:, 40] = 0
    assert np.isfinite(got).all()
    if dtype == "bf16":
        assert (f64(G)[:, 40] == np.inf).all()

"""Products of at most 16 rows: every share of the weights' rows that a workgroup can
take (8 at least, up to 16 in one MFMA's rows and 32 in two, in one round of workgroups
and in several), its last workgroup with fewer, and one row past the limit."""

import numpy as np
import pytest

from layer_helpers import say
from matrix_optimizer_step_muon_amd import layer
from product_helpers import Mlp
from test_linear8_gpu import Item, run

pytestmark = pytest.mark.gpu

# 256 CUs: 8 rows of weights up to 2048 of them, 9 from 2049, 16 up to 4096, 17 to 32 up
# to 8192, then two rounds (in fp32 from 4097).
WIDE = [7, 2047, 2049, 4096, 4097, 5120, 6140, 8192, 8193, 12001, 16400]


@pytest.mark.parametrize("rows", [1, 5, 16, 17])
@pytest.mark.parametrize("n", WIDE)
def test_shares_of_8_bit_weights(rows, n):
    say(rows, n)
    run(Item(rows, n, 300, "bf16", beta=0.5))
    run(Item(rows, 140, n, "bf16", transposed=True, ld=3, offset=1))


@pytest.mark.parametrize("rows", [1, 16])
@pytest.mark.parametrize("k", [1, 127, 128, 129, 255, 256, 257, 2048, 2049, 4095, 4100, 8191])
def test_lengths_of_8_bit_sums(rows, k):
    say(rows, k)
    run(Item(rows, 40, k, "bf16"))
    run(Item(rows, 4100, k, "bf16") if k <= 2049 else Item(rows, 40, k, "bf16", beta=1.0, own_c=False))


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("bf16", "relu"), ("f32", "gelu")])
@pytest.mark.parametrize("rows", [1, 16, 17])
@pytest.mark.parametrize("n", WIDE)
def test_shares_of_the_gated_blocks_weights(rows, n, dtype, act):
    say(rows, n, dtype, act)
    for m in (Mlp(rows, 136, n, 24, dtype, act, None, seed=rows + n), Mlp(rows, 24, 72, n, dtype, act, None, seed=rows + n)):
        m.forward()
        m.check_forward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1023, 1025, 2047, 2049])
def test_lengths_of_the_gated_blocks_sums(dtype, k):
    say(dtype, k)
    for m in (Mlp(3, k, 40, 24, dtype, "silu", None, seed=k), Mlp(3, 24, k, 40, dtype, "silu", None, seed=k)):
        m.forward()
        m.check_forward()


def test_items_without_rows_beside_others():
    import torch
    w = layer.W8(64, 96)
    layer.w8_save(torch.ones(64, 96, device="cuda"), w)
    none = (layer.Q8(0, 96, "e4m3"), w, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    layer.Linear8([none]).run()
    few, many = Item(4, 64, 96, "bf16"), Item(40, 64, 96, "bf16")
    layer.Linear8([none, few.item, none, many.item]).run()
    for i in (few, many):
        i.check()
    assert np.all(w.e.cpu().numpy() > 0)

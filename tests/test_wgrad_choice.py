"""Which of the weight gradient's kernels a product takes, and every kernel with
its sum whole and in pieces against the fp64 oracle. Each case names the tile
and the pieces it is here for, so that another choice fails instead of moving
the coverage elsewhere. Tolerances as in test_wgrad_gpu.py."""

import ctypes

import pytest

from matrix_optimizer_step_muon_amd import muon

BASE, STEP = 0x7F0000000000, 1 << 34
PARTS = {"bf16": muon.MUON_BF16, "f32": muon.MUON_F32}

# rows, n, k, dtype, gdtype, kind, tile, pieces. fp32 sums over three planes of
# rows one after the other: two and four pieces start inside a plane.
WHOLE = [
    (300, 1000, 1100, "bf16", "f32", "int8", 64, 1), (150, 1001, 1101, "f32", "f32", "e4m3", 64, 1),
    (1000, 2048, 4096, "bf16", "f32", "e4m3", 128, 1), (260, 2560, 2500, "f32", "f32", "int8", 128, 1),
    (520, 2500, 2560, "f32", "bf16", "e4m3", 128, 1),
    (700, 2100, 4099, "bf16", "f32", "int8", 256, 1), (1000, 4096, 4200, "bf16", "bf16", "e4m3", 256, 1),
    (1000, 4097, 4200, "f32", "f32", "int8", 256, 1),
]
CUT = [
    (3001, 40, 264, "bf16", "f32", "int8", 64, 12), (300, 48, 64, "f32", "f32", "e4m3", 64, 3),
    (2700, 1024, 1030, "bf16", "f32", "int8", 128, 3), (4095, 260, 5300, "f32", "f32", "e4m3", 128, 4),
    (4096, 1024, 5120, "bf16", "f32", "int8", 256, 3), (4097, 1023, 5121, "bf16", "bf16", "e4m3", 256, 3),
    (3000, 1032, 5100, "bf16", "f32", "e4m3", 256, 2), (3000, 1031, 5100, "f32", "f32", "int8", 256, 2),
    (8191, 520, 5120, "f32", "f32", "e4m3", 256, 4), (5000, 1001, 5003, "f32", "bf16", "int8", 256, 3),
]


def described(sizes, dtype, kind=0):
    """Items at made-up addresses, which nothing dereferences."""
    items = (muon.muon_wgrad_item * len(sizes))()
    for i, (rows, n, k) in enumerate(sizes):
        a = BASE + 8 * i * STEP
        x = muon.muon_q8(a + STEP, a + 2 * STEP, rows, k, -(-k // 16) * 16, -(-k // 32), kind, 0)
        items[i] = muon.muon_wgrad_item(a, n, x, None, a + 3 * STEP, a + 4 * STEP, n, 0.0, 0)
    return items


def info(items, dtype, gdtype="f32"):
    n = len(items)
    tile, pieces = (ctypes.c_int32 * n)(), (ctypes.c_int32 * n)()
    muon.check(muon.lib().muon_wgrad_info(items, n, PARTS[dtype], PARTS[gdtype], tile, pieces))
    return list(zip(tile, pieces))


@pytest.mark.parametrize("rows,n,k,dtype,gdtype,kind,tile,pieces", WHOLE + CUT)
def test_the_cases_take_the_kernels_they_are_here_for(rows, n, k, dtype, gdtype, kind, tile, pieces):
    items = described([(rows, n, k)], dtype)
    assert info(items, dtype, gdtype) == [(tile, pieces)]
    need = ctypes.c_size_t()
    muon.check(muon.lib().muon_wgrad_workspace(items, 1, PARTS[dtype], PARTS[gdtype], ctypes.byref(need)))
    tiles = -(-n // tile) * -(-k // tile)
    partial = tiles * pieces * tile * tile * 4 if pieces > 1 else 0
    planes = 0 if tile == 64 else 3 if dtype == "f32" else n % 8 != 0
    packed = -(-(planes * rows * -(-n // 8) * 8 * 2) // 256) * 256
    assert need.value == partial + packed


def test_items_past_one_launch_and_without_rows():
    # 16 items share a launch and its tile; each item has pieces of its own
    sizes = [(4096, 1024, 5120)] * 16 + [(0, 40, 50), (1, 64, 64)]
    got = info(described(sizes, "bf16"), "bf16")
    assert {t for t, _ in got[:16]} == {256} and {t for t, _ in got[16:]} == {64}
    assert got[16][1] == 1 and got[17][1] == 1


def test_refusals():
    L, one = muon.lib(), described([(40, 64, 100)], "bf16")
    t, p = ctypes.c_int32(), ctypes.c_int32()
    for args in ((one, 1, 1, 1, None, ctypes.byref(p)), (one, 1, 1, 1, ctypes.byref(t), None), (None, 1, 1, 1, ctypes.byref(t), ctypes.byref(p)),
                 (one, 0, 1, 1, ctypes.byref(t), ctypes.byref(p))):
        assert L.muon_wgrad_info(*args) == -1
    assert L.muon_wgrad_info(one, 1, 2, 1, ctypes.byref(t), ctypes.byref(p)) == -4
    one[0].g = one[0].dy
    assert L.muon_wgrad_info(one, 1, 1, 1, ctypes.byref(t), ctypes.byref(p)) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k,dtype,gdtype,kind,tile,pieces", WHOLE + CUT)
def test_product(rows, n, k, dtype, gdtype, kind, tile, pieces):
    import torch

    from layer_helpers import say
    from matrix_optimizer_step_muon_amd import layer
    from test_wgrad_gpu import Item
    say("case", rows, n, k, dtype, gdtype, kind)
    it = Item(rows, n, k, dtype, gdtype, kind, scale=k % 2 == 0, beta=1.0 if n % 2 == 0 else 0.0, own_c=rows % 2 == 1, seed=rows)
    plan = layer.WGrad([it.item])
    assert plan.info() == [{"tile": tile, "pieces": pieces}]
    plan.run()
    torch.cuda.synchronize()
    it.check()
    if it.beta == 0:
        first = it.G.clone()
        it.G.fill_(3.0)
        plan.run()
        torch.cuda.synchronize()
        assert torch.equal(first, it.G), "the same call twice gives other bits"

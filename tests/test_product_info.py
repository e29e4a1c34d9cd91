"""How the layers' products say they are cut up, without a GPU."""

import ctypes

import pytest

from matrix_optimizer_step_muon_amd import muon
from test_product_abi import L, grads, item, last, mlp


def cuts(f, *args, n=2):
    t = [(ctypes.c_int32 * n)() for _ in range(3)]
    assert f(*args, *t) == 0, muon.last_error()
    return [tuple(x[i] for x in t) for i in range(n)]


def tiles(rows, cols, edge):
    return -(-rows // edge) * -(-cols // edge)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,width,inner,out", [(40, 64, 100, 72), (300, 2048, 6144, 2048), (4096, 2048, 6144, 2048), (4100, 4360, 4368, 4360)])
def test_blocks(rows, width, inner, out, dtype):
    """Whole tiles are at most all of a product, and pieces are only of what is left."""
    m, g = mlp(rows, width, inner, out, dtype=dtype), grads(width, inner, out)
    both = cuts(L.muon_mlp_info, m, None) + cuts(L.muon_mlp_info, m, g)
    for (tile, whole, pieces), cols, sides in zip(both, (inner, out, inner, width), (2, 1, 1, 1)):
        assert tile in (64, 128, 256)
        count = -(-rows // tile) * -(-cols * sides // tile) if sides == 1 else -(-rows // tile) * -(-cols // (tile // 2))
        assert (whole == count and pieces == 1) or (whole < count and 2 <= pieces <= 64)


def test_what_is_not_made_and_few_rows():
    m, g = mlp(), grads()
    m.y = g.d_x = None
    assert cuts(L.muon_mlp_info, m, None)[1] == (0, 0, 1) and cuts(L.muon_mlp_info, m, g)[1] == (0, 0, 1)
    few = mlp(1, 2048, 6144, 2048)
    few.a = few.b = few.s = muon.muon_q8()
    assert cuts(L.muon_mlp_info, few, None) == [(0, 0, 1)] * 2
    assert cuts(L.muon_mlp_info, mlp(rows=0), g) == [(0, 0, 1)] * 2
    items = (muon.muon_linear8_item * 3)(item(0, rows=16), item(1, rows=17), item(2, rows=200))
    first, *others = cuts(L.muon_linear8_info, items, 3, 1, n=3)
    edge = others[0][0]
    assert first == (0, 0, 1) and edge > 0 and others == [(edge, tiles(r, 72, edge), 1) for r in (17, 200)]
    assert cuts(L.muon_linear8_info, items, 3, 0, n=3)[0][0] > 0     # fp32 results come from tiles


def test_more_items_than_a_launch_holds():
    """Items that go in tiles are numbered past those of few rows, 16 to a launch, each
    of which has one size of tiles."""
    n = 60
    items = (muon.muon_linear8_item * n)(*[item(i, rows=16 if i % 3 else 200 * (i + 1)) for i in range(n)])
    got = cuts(L.muon_linear8_info, items, n, 1, n=n)
    for i, (tile, whole, pieces) in enumerate(got):
        if i % 3:
            assert (tile, whole, pieces) == (0, 0, 1), i
        else:
            assert tile == got[0 if i < 48 else 48][0] > 0 and pieces == 1 and whole == tiles(200 * (i + 1), 72, tile), (i, got[i])


def test_refusals():
    t = [(ctypes.c_int32 * 2)() for _ in range(3)]
    for bad in range(3):
        args = [None if i == bad else x for i, x in enumerate(t)]
        assert L.muon_mlp_info(mlp(), None, *args) == -1 and L.muon_linear8_info(item(), 1, 1, *args) == -1
    assert L.muon_mlp_info(None, None, *t) == -1
    last(L.muon_mlp_info(mlp(width=0), None, *t), -1, "width")
    last(L.muon_linear8_info(None, 1, 1, *t), -1, "items is NULL")
    it = item()
    it.x.kind = 0
    last(L.muon_linear8_info(it, 1, 1, *t), -4, "e4m3")

"""fp32 blocks to fp32 accuracy, in norm: the bounds by element are for the worst case,
which for a sum of 2000 terms is a hundred times what its roundings come to. Every size
of tile in both orientations, and the kernels for few rows."""

import numpy as np
import pytest

from layer_helpers import codes, f64, say
from oracle import layer_ref, product_ref as ref
from product_helpers import Mlp
from test_fp32_parts import NORM

pytestmark = pytest.mark.gpu


def sync():
    import torch
    torch.cuda.synchronize()


def close(got, want, what):
    e = np.linalg.norm(got - want) / np.linalg.norm(want)
    say(what, f"{e:.2e}")
    assert e < NORM, what


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("rows", [1, 5, 16])
@pytest.mark.parametrize("width,inner,out", [(500, 1000, 72), (2048, 500, 264), (1000, 2048, 500)])
def test_few_rows(rows, width, inner, out, act):
    m = Mlp(rows, width, inner, out, "f32", act, None, seed=rows + width)
    assert [c["tile"] for c in m.mlp.info()["forward"]] == [0, 0]
    m.forward()
    sync()
    close(f64(m.mlp.y), ref.mlp_forward(m.x, m.wg, m.wu, m.wd, act)[3], "y")


TILES = [  # rows, width, inner, out; the tiles of a/b, y, ds, d_x
    (20, 500, 500, 500, (64, 64, 64, 64)), (600, 1000, 1000, 500, (128, 64, 64, 128)), (1024, 500, 1000, 1000, (64, 64, 128, 64)),
    (600, 1000, 1000, 2048, (128, 128, 128, 128)), (1500, 1000, 1000, 2048, (256, 256, 256, 256)),
]


@pytest.mark.parametrize("rows,width,inner,out,tiles", TILES)
def test_tiles(rows, width, inner, out, tiles):
    act = "silu"
    m = Mlp(rows, width, inner, out, "f32", act, "int8", seed=rows + out)
    cuts = m.mlp.info()
    assert tuple(c["tile"] for c in cuts["forward"] + cuts["backward"]) == tiles, cuts
    m.forward().backward()
    sync()
    close(f64(m.mlp.y), ref.mlp_forward(m.x, m.wg, m.wu, m.wd, act)[3], "y")
    a, b = (layer_ref.q8_decode(*codes(q), "int8") for q in (m.mlp.a, m.mlp.b))
    _, da, db, dx = ref.mlp_backward(m.dy, a, b, m.wg, m.wu, m.wd, act)
    for name, want in (("d_a", da), ("d_b", db), ("d_x", dx)):
        close(f64(getattr(m.mlp, name)), want, name)

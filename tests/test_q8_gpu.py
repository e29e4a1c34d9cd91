"""8-bit checkpoints against the fp64 oracle, bit for bit: the scales are powers
of two, so every code has one right value."""

import numpy as np
import pytest

from layer_helpers import codes, dev, device_q8, f64, rng, say, stored, tdt
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu


def activations(rows, cols, seed):
    g = rng(seed)
    x = g.standard_normal((rows, cols)) * np.exp(3 * g.standard_normal((rows, 1)))
    return x * np.where(g.random(cols) < 0.05, 100.0, 1.0)


def round_trip(x, dtype, kind, **view):
    import torch
    xs = stored(x, dtype)
    t = dev(x, dtype, **view)
    ckpt = layer.Q8(x.shape[0], x.shape[1], kind)
    ckpt.q.fill_(0x55)
    layer.q8_save(t, ckpt)
    outs = {}
    for od in ("bf16", "f32"):
        outs[od] = torch.full(x.shape, 7.0, dtype=tdt(od), device="cuda")
        layer.q8_load(ckpt, outs[od])
    torch.cuda.synchronize()
    q, e = codes(ckpt)
    wq, we = ref.q8_encode(xs, kind)
    assert np.array_equal(e, we), "exponent bytes"
    assert np.array_equal(q, wq), "codes"
    want = ref.q8_decode(wq, we, kind)
    for od, t in outs.items():
        assert np.array_equal(f64(t), want, equal_nan=True), f"loaded {od}"
    return want


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (5, 33), (2, 200), (7, 64), (9, 1111), (1, 5120), (300, 40)])
def test_round_trip(rows, cols, dtype, kind):
    say("case", rows, cols, dtype, kind)
    round_trip(activations(rows, cols, rows * 10007 + cols), dtype, kind)


@pytest.mark.parametrize("ld,offset", [(131, 0), (144, 3), (136, 8), (129, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_unaligned_input(ld, offset, dtype):
    say("case", ld, offset, dtype)
    round_trip(activations(6, 128, ld), dtype, "int8", ld=ld, offset=offset)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_borders_of_the_format(kind):
    # The largest magnitude exactly at, just below and just above a power of two
    # and the top of the grid; ties; zeros of both signs; tiny and huge values.
    top = ref.TOP[kind]
    rows = []
    for k in (-130, -112, -111, -110, -5, 0, 7, 100, 118):
        for m in (top, top * (1 + 2.0 ** -23), top * (1 - 2.0 ** -23), 64.0, 128.0, 1.0):
            v = np.zeros(40)
            v[0] = m * 2.0 ** k
            v[1:9] = np.array([0.5, 1.5, 2.5, -0.5, -1.5, 3.5, 0.25, -0.0]) * 2.0 ** k
            v[9:17] = np.array([17, 19, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -7]) * 2.0 ** k
            v[32] = -m * 2.0 ** k
            rows.append(v)
    x = np.array(rows)
    x = x[np.isfinite(x.astype(np.float32)).all(1)]
    round_trip(x, "f32", kind)
    round_trip(x, "bf16", kind)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_non_finite_groups_stand_for_nan(kind):
    x = activations(6, 100, 3)
    x[0, 5], x[1, 40], x[2, 99], x[3, 96], x[4, 31] = np.inf, -np.inf, np.nan, np.inf, np.nan
    want = round_trip(x, "f32", kind)
    assert np.isnan(want[0, :32]).all() and np.isfinite(want[0, 32:]).all()
    assert np.isnan(want[2, 96:]).all() and np.isfinite(want[5]).all()


def test_no_rows():
    import torch
    ckpt = layer.Q8(0, 50)
    layer.q8_save(torch.empty(0, 50, device="cuda"), ckpt)
    layer.q8_load(ckpt, torch.empty(0, 50, device="cuda"))
    torch.cuda.synchronize()


def test_views_of_wider_checkpoints_leave_the_rest_alone():
    import torch
    x = activations(5, 96, 8)
    q = torch.full((5, 160), 0xAB, dtype=torch.uint8, device="cuda")
    e = torch.full((5, 7), 0xCD, dtype=torch.uint8, device="cuda")
    ckpt = layer.Q8(5, 96, "int8", q=q[:, 32:], e=e[:, 2:])
    layer.q8_save(dev(x, "f32"), ckpt)
    torch.cuda.synchronize()
    wq, we = ref.q8_encode(stored(x, "f32"), "int8")
    assert np.array_equal(q[:, 32:128].cpu().numpy(), wq) and np.array_equal(e[:, 2:5].cpu().numpy(), we)
    assert (q[:, :32] == 0xAB).all() and (q[:, 128:] == 0xAB).all()
    assert (e[:, :2] == 0xCD).all() and (e[:, 5:] == 0xCD).all()
    out = torch.full((5, 100), 3.0, device="cuda")
    layer.q8_load(device_q8(wq, we, "int8"), out[:, 2:98])
    torch.cuda.synchronize()
    assert np.array_equal(f64(out[:, 2:98]), ref.q8_decode(wq, we, "int8"))
    assert (out[:, :2] == 3).all() and (out[:, 98:] == 3).all()

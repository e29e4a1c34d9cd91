"""Norm sites against the fp64 oracle, forward and backward.

Tolerances. An output is rounded once to its type (HALF of its value). Before
that, fp32: every value is a sum of a few terms, each a product of a few
factors, and row means are trees of at most 8 + 6 + 16 + 4 additions; DEPTH
fp32 roundings of the terms' magnitudes cover both. A weight gradient adds at
most 16 + 64 + 16 partial sums after that, one rounding each, and rows of the
test cases / 256 in a workgroup.
"""

import numpy as np
import pytest

from layer_helpers import F32, HALF, codes, dev, device_q8, f64, rng, say, stored, tdt, within
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu
DEPTH = 48
EPS = 1e-6


def make(rows, cols, dtype, post, gate, seed):
    g = rng(seed)
    d = {"b": g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1))),
         "r": g.standard_normal((rows, cols)), "w_pre": 1 + 0.3 * g.standard_normal(cols),
         "w_post": 1 + 0.3 * g.standard_normal(cols) if post else None,
         "gate": None if gate == "none" else g.standard_normal(cols if gate == "feature" else (rows, cols)),
         "dy": 1e-3 * g.standard_normal((rows, cols)), "dh": 1e-3 * g.standard_normal((rows, cols))}
    return {k: None if v is None else stored(v, dtype) for k, v in d.items()}


def site_of(d, dtype, kind, saved=None, **view):
    t = {k: None if d[k] is None else dev(d[k], dtype, **(view if d[k].ndim == 2 else {})) for k in ("b", "r", "w_pre", "w_post", "gate")}
    return layer.NormSite(t["b"], t["r"], t["w_pre"], w_post=t["w_post"], gate=t["gate"], res_scale=0.75, branch_scale=1.25,
                          eps=EPS, kind=kind, saved=saved)


def forward_want(d):
    return ref.norm_forward(d["b"], d["r"], d["w_pre"], d["w_post"], d["gate"], 0.75, 1.25, EPS)


def magnitudes(d, rstd_b):
    n = np.abs(d["b"]) * rstd_b[:, None]
    for w in (d["w_post"], d["gate"]):
        n = n if w is None else n * np.abs(w)
    return 0.75 * np.abs(d["r"]) + 1.25 * n


def check_forward(site, d, dtype, kind):
    y, h, u, v, ry, rb = forward_want(d)
    m = magnitudes(d, rb)
    within(f64(site.y), y, HALF[dtype] * np.abs(y) + DEPTH * F32 * m, "y")
    mu = m * ry[:, None]
    within(f64(site.h), h, HALF[dtype] * np.abs(h) + DEPTH * F32 * np.abs(d["w_pre"]) * mu, "h")
    if kind is None:
        return
    within(f64(site.rstd_y), ry, DEPTH * F32 * ry, "rstd_y")
    if d["w_post"] is not None:
        within(f64(site.rstd_b), rb, DEPTH * F32 * rb, "rstd_b")
    for name, ckpt, want, mag in (("u", site.u, u, mu), ("v", site.v, v, np.abs(v))):
        if ckpt is None:
            continue
        q, e = codes(ckpt)
        got = ref.q8_decode(q, e, kind)
        unit = np.repeat(2.0 ** (e.astype(float) - 127), 32, axis=1)[:, :want.shape[1]]
        # the grid: the smallest that holds the group's largest magnitude
        cols = want.shape[1]
        for g in range(e.shape[1]):
            s = slice(32 * g, min(32 * g + 32, cols))
            top, slack = np.abs(want[:, s]).max(1), DEPTH * F32 * mag[:, s].max(1)
            k = 2.0 ** (e[:, g].astype(float) - 127)
            assert (top - slack <= ref.TOP[kind] * k).all() and (top + slack > ref.TOP[kind] * k / 2).all(), f"{name}: exponents"
        # half a step of the grid: 1/2 for int8; 2^-4 of the value, or 2^-10 below 2^-6, for e4m3
        half = 0.5 * unit if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * unit)
        within(got, want, half * (1 + 1e-6) + DEPTH * F32 * mag, name)


def check_backward(site, d, u, v, ry, rb, dtype, dy_none=False):
    dy = np.zeros_like(d["dy"]) if dy_none else d["dy"]
    args = (u, v, ry, rb, d["w_pre"], d["w_post"], d["gate"], 0.75, 1.25)
    want = ref.norm_backward(dy, d["dh"], *args)
    a = np.abs
    # magnitudes: the same sums with every term positive
    du = a(d["dh"] * d["w_pre"])
    ms = a(dy) + ry[:, None] * (du + a(u) * (du * a(u)).mean(1, keepdims=True))
    w2, gt = (1.0 if d["w_post"] is None else a(d["w_post"])), (1.0 if d["gate"] is None else a(d["gate"]))
    mb = 1.25 * ms * gt * w2
    if d["w_post"] is not None:
        mb = rb[:, None] * (mb + a(v) * (mb * a(v)).mean(1, keepdims=True))
    rows = len(u)
    more = DEPTH + 96 + rows / 256
    within(f64(site.d_residual), want[0], HALF[dtype] * a(want[0]) + DEPTH * F32 * 0.75 * ms, "d_residual")
    within(f64(site.d_branch), want[1], HALF[dtype] * a(want[1]) + 2 * DEPTH * F32 * mb, "d_branch")
    within(f64(site.d_w_pre), want[2], HALF[dtype] * a(want[2]) + more * F32 * a(d["dh"] * u).sum(0), "d_w_pre")
    if d["w_post"] is not None:
        within(f64(site.d_w_post), want[3], HALF[dtype] * a(want[3]) + more * F32 * (1.25 * ms * gt * a(v)).sum(0), "d_w_post")
    else:
        assert site.d_w_post is None
    if d["gate"] is not None:
        mg = 1.25 * ms * w2 * a(v)
        mg = mg if d["gate"].ndim == 2 else mg.sum(0)
        within(f64(site.d_gate), want[4], HALF[dtype] * a(want[4]) + more * F32 * mg, "d_gate")
    else:
        assert site.d_gate is None


CASES = [  # rows, cols, post, gate
    (1, 1, True, "feature"), (1, 32, False, "none"), (3, 31, True, "token"), (5, 200, True, "none"),
    (7, 512, False, "feature"), (4, 513, True, "feature"), (2, 2048, True, "token"), (3, 5120, True, "feature"),
    (2, 8192, True, "feature"), (2, 8200, False, "token"), (1, 16384, True, "feature"), (2, 16391, True, "token"),
    (1, 32768, True, "none"), (700, 64, True, "feature"), (3000, 40, True, "feature"), (1500, 33, False, "feature"),
]


@pytest.mark.parametrize("dtype,kind", [("bf16", "int8"), ("bf16", "e4m3"), ("f32", "int8"), ("f32", None)])
@pytest.mark.parametrize("rows,cols,post,gate", CASES)
def test_forward(rows, cols, post, gate, dtype, kind):
    import torch
    say("case", rows, cols, post, gate, dtype, kind)
    d = make(rows, cols, dtype, post, gate, rows + cols)
    site = site_of(d, dtype, kind)
    site.y.fill_(float("nan"))
    site.h.fill_(float("nan"))
    site.forward()
    torch.cuda.synchronize()
    check_forward(site, d, dtype, kind)


@pytest.mark.parametrize("dtype,kind", [("bf16", "int8"), ("f32", "e4m3")])
@pytest.mark.parametrize("rows,cols,post,gate", CASES)
def test_backward_from_given_checkpoints(rows, cols, post, gate, dtype, kind):
    import torch
    say("case", rows, cols, post, gate, dtype, kind)
    d = make(rows, cols, dtype, post, gate, rows + cols)
    _, _, u, v, ry, rb = forward_want(d)
    ry, rb = stored(ry, "f32"), stored(rb, "f32")
    (qu, eu), (qv, ev) = _encode_fast(u, kind), _encode_fast(v, kind)
    u, v = ref.q8_decode(qu, eu, kind), ref.q8_decode(qv, ev, kind)
    site = site_of(d, dtype, kind, saved=(device_q8(qu, eu, kind), device_q8(qv, ev, kind), dev(ry, "f32"), dev(rb, "f32")))
    site.backward(dev(d["dy"], dtype), dev(d["dh"], dtype))
    torch.cuda.synchronize()
    check_backward(site, d, u, v, ry, rb, dtype)
    first = [t.clone() for t in (site.d_residual, site.d_branch, site.d_w_pre)]
    site.backward(dev(d["dy"], dtype), dev(d["dh"], dtype))
    torch.cuda.synchronize()
    for x, y in zip(first, (site.d_residual, site.d_branch, site.d_w_pre)):
        assert torch.equal(x, y), "the same call twice gives other bits"


def _encode_fast(x, kind):
    """Codes of x; the oracle's encoder is a loop, so large inputs take its first rows many times."""
    return ref.q8_encode(x, kind) if x.size < 200000 else _stack(x, kind)


def _stack(x, kind):
    parts = [ref.q8_encode(x[i:i + 1000], kind) for i in range(0, len(x), 1000)]
    return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_backward_reads_what_the_forward_kept(kind):
    import torch
    d = make(50, 333, "bf16", True, "token", 5)
    site = site_of(d, "bf16", kind)
    site.forward()
    site.backward(None, dev(d["dh"], "bf16"))
    torch.cuda.synchronize()
    u, v = (ref.q8_decode(*codes(c), kind) for c in (site.u, site.v))
    check_backward(site, d, u, v, f64(site.rstd_y), f64(site.rstd_b), "bf16", dy_none=True)


@pytest.mark.parametrize("ld,offset", [(101, 0), (112, 8), (107, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_unaligned_views(ld, offset, dtype):
    import torch
    say("case", ld, offset, dtype)
    d = make(9, 96, dtype, True, "token", 11)
    site = site_of(d, dtype, "int8", ld=ld, offset=offset)
    site.forward()
    site.backward(dev(d["dy"], dtype, ld=ld, offset=offset), dev(d["dh"], dtype, ld=ld, offset=offset))
    torch.cuda.synchronize()
    check_forward(site, d, dtype, "int8")
    u, v = (ref.q8_decode(*codes(c), "int8") for c in (site.u, site.v))
    check_backward(site, d, u, v, f64(site.rstd_y), f64(site.rstd_b), dtype)


def test_no_rows_gives_zero_weight_gradients():
    import torch
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    site = layer.NormSite(z(0, 70), z(0, 70), torch.ones(70, device="cuda"), w_post=z(70), gate=z(70))
    site.forward()
    site.backward(z(0, 70), z(0, 70))
    site.d_w_pre.fill_(5.0)
    site.backward(z(0, 70), z(0, 70))
    torch.cuda.synchronize()
    assert not site.d_w_pre.any() and not site.d_w_post.any() and not site.d_gate.any()


def test_zero_rows_and_non_finite_rows_stay_in_their_row():
    import torch
    d = make(6, 128, "f32", True, "feature", 3)
    d["b"][1], d["r"][1] = 0.0, 0.0      # norms of zero: 1/sqrt(eps), finite
    d["b"][2, 7], d["r"][4, 100] = np.nan, np.inf
    site = site_of(d, "f32", "int8")
    site.forward()
    site.backward(dev(d["dy"], "f32"), dev(d["dh"], "f32"))
    torch.cuda.synchronize()
    y, h = f64(site.y), f64(site.h)
    assert not y[1].any() and not h[1].any()
    assert np.isnan(h[2]).all() and not np.isfinite(h[4, 100])
    dr, db = f64(site.d_residual), f64(site.d_branch)
    for r in (0, 1, 3, 5):
        assert np.isfinite(y[r]).all() and np.isfinite(h[r]).all() and np.isfinite(dr[r]).all() and np.isfinite(db[r]).all()
    assert np.isnan(dr[2]).all() and np.isnan(dr[4]).all(), "a bad activation shows up in the gradient"
    assert np.isnan(f64(site.d_w_pre)).any()


def test_gradients_against_differences():
    # d/dx of sum(dy*y + dh*h) by central differences of the fp64 forward, against
    # the kernel's gradients in fp32. The checkpoints' rounding (2^-7 of a
    # group's top per element for int8, at worst) bounds the difference.
    import torch
    d = make(4, 64, "f32", True, "feature", 21)
    site = site_of(d, "f32", "int8")
    site.forward()
    site.backward(dev(d["dy"], "f32"), dev(d["dh"], "f32"))
    torch.cuda.synchronize()

    def loss(x):
        y, h, *_ = forward_want(x)
        return (d["dy"] * y).sum() + (d["dh"] * h).sum()

    g = rng(1)
    for name, grad in (("b", site.d_branch), ("r", site.d_residual), ("w_pre", site.d_w_pre), ("w_post", site.d_w_post),
                       ("gate", site.d_gate)):
        t = g.standard_normal(d[name].shape)
        e = 1e-5
        diff = (loss({**d, name: d[name] + e * t}) - loss({**d, name: d[name] - e * t})) / (2 * e)
        got = f64(grad)
        # a random direction: the error of a gradient with relative error 2^-6 (two checkpoints), four sigma
        assert abs((got * t).sum() - diff) <= 4 * 2.0 ** -6 * np.linalg.norm(got), name


def test_another_stream_and_graph_replays():
    import torch
    d = make(64, 256, "bf16", True, "feature", 9)
    site = site_of(d, "bf16", "int8")
    dy, dh = dev(d["dy"], "bf16"), dev(d["dh"], "bf16")
    site.forward()
    site.backward(dy, dh)
    torch.cuda.synchronize()
    names = ("y", "h", "d_residual", "d_branch", "d_w_pre", "d_w_post", "d_gate")
    want = {n: getattr(site, n).clone() for n in names}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for n in names:
        getattr(site, n).zero_()
    side.wait_stream(torch.cuda.current_stream())
    site.forward(side)
    site.backward(dy, dh, side)
    side.synchronize()
    for n in names:
        assert torch.equal(getattr(site, n), want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        site.forward()
        site.backward(dy, dh)
    for _ in range(3):
        for n in names:
            getattr(site, n).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(getattr(site, n), want[n]), n
        site.forward()
        site.backward(dy, dh)
        torch.cuda.synchronize()

"""The gated feed-forward block against the fp64 oracle; the bounds are those of
product_helpers."""

import numpy as np
import pytest

from layer_helpers import HALF, dev, f64, say, tdt
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref, product_ref as ref
from product_helpers import Mlp

pytestmark = pytest.mark.gpu


def sync():
    import torch
    torch.cuda.synchronize()


def both(m, what=""):
    say(what, m.rows, m.x.shape, m.wg.shape, m.wd.shape, m.dtype, m.act, m.kind)
    m.forward().backward()
    sync()
    m.check_forward(what)
    m.check_backward(what)


SIZES = [  # rows, width, inner, out
    (1, 1, 1, 1), (1, 128, 256, 128), (2, 8, 16, 8), (5, 33, 77, 19), (16, 64, 64, 64), (17, 65, 130, 66), (63, 72, 96, 200),
    (64, 128, 64, 64), (65, 200, 264, 136), (130, 201, 333, 97), (200, 520, 40, 1100), (300, 24, 700, 8), (257, 136, 512, 264),
]


@pytest.mark.parametrize("dtype,kind,act", [("bf16", "int8", "silu"), ("bf16", "e4m3", "gelu"), ("f32", "int8", "gelu_tanh"),
                                            ("f32", "e4m3", "relu")])
@pytest.mark.parametrize("rows,width,inner,out", SIZES)
def test_sizes(rows, width, inner, out, dtype, kind, act):
    both(Mlp(rows, width, inner, out, dtype, act, kind, seed=rows + inner))


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activations_over_their_range(act, dtype):
    """Gate sums from -40 to 40: where the activation is curved, flat and saturated."""
    def edit(m):
        m.x[:] = 0
        m.x[:, 0] = np.linspace(-40, 40, m.rows)
        m.wg[:] = 0
        m.wg[:, 0] = 1
        m.x[:] = np.float32(m.x)
        if dtype == "bf16":
            import torch
            m.x[:] = torch.from_numpy(m.x).to(torch.bfloat16).double().numpy()
    both(Mlp(160, 40, 64, 32, dtype, act, "int8", seed=3, edit=edit))


@pytest.mark.parametrize("rows", [1, 3, 16])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f32", "gelu")])
@pytest.mark.parametrize("width,inner,out", [(2048, 640, 520), (129, 1000, 33), (7, 16, 2000), (640, 17, 16), (1100, 33, 513)])
def test_few_rows_that_keep_nothing(rows, width, inner, out, dtype, act):
    m = Mlp(rows, width, inner, out, dtype, act, None, seed=rows + out)
    say(rows, width, inner, out, dtype)
    m.forward()
    sync()
    m.check_forward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 100])
@pytest.mark.parametrize("ld,offset,weight_offset", [(8, 8, 0), (3, 1, 0), (0, 0, 1), (5, 3, 7)])
def test_views_and_alignments(dtype, rows, ld, offset, weight_offset):
    for kind in ("int8", None):
        m = Mlp(rows, 96, 160, 64, dtype, "silu", kind, seed=7, ld=ld, offset=offset, weight_offset=weight_offset)
        m.forward()
        sync()
        m.check_forward()
        if kind:
            m.backward()
            sync()
            m.check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,shift", [(3, 0), (70, 0), (70, 5), (300, 8)])
def test_the_output_may_be_a_view_and_nothing_around_it_is_written(rows, shift, dtype):
    import torch
    buf = torch.full((rows + 4, 100), -77.0, dtype=tdt(dtype), device="cuda")
    y = buf[2:2 + rows, shift:shift + 72]
    m = Mlp(rows, 64, 136, 72, dtype, "silu", None, seed=5, out_tensor=y)
    m.forward()
    sync()
    m.check_forward()
    buf[2:2 + rows, shift:shift + 72] = -77.0
    assert (buf == -77).all()


def test_more_rounds_of_tiles_than_cus_and_pieces():
    """Sizes that take large tiles, whole and in pieces, and a last round in pieces."""
    for rows, width, inner, out in ((2048, 384, 4352, 384), (1030, 1000, 2056, 520), (520, 4096, 264, 1032)):
        both(Mlp(rows, width, inner, out, "bf16", "silu", "int8", seed=rows))


def test_fp32_in_large_tiles():
    both(Mlp(1100, 264, 1032, 528, "f32", "silu", "int8", seed=9))


def test_checkpoints_one_by_one():
    """Each may be left out; what is kept does not depend on the others: a and b bit for
    bit, s but for a last bit of its fp32 value, which may cross a rounding border (one
    step of its code, and of the row's sum its own bound)."""
    import torch
    m = Mlp(200, 136, 264, 72, "bf16", "silu", "int8", seed=1)
    m.forward()
    sync()
    whole = [(q.q.clone(), q.e.clone()) for q in (m.mlp.a, m.mlp.b, m.mlp.s)]
    y = m.mlp.y.clone()
    c = m.mlp._c
    saved = [c.a.q, c.b.q, c.s.q]
    for keep in range(1, 8):
        for q in (m.mlp.a, m.mlp.b, m.mlp.s):
            q.q.fill_(1)
            q.e.fill_(1)
        c.a.q, c.b.q, c.s.q = (p if keep >> i & 1 else None for i, p in enumerate(saved))
        m.mlp.forward()
        sync()
        for i, q in enumerate((m.mlp.a, m.mlp.b, m.mlp.s)):
            if not keep >> i & 1:
                assert bool((q.q == 1).all()) and bool((q.e == 1).all()), (keep, i)
            elif i < 2:
                assert bool((q.q[:, :264] == whole[i][0][:, :264]).all()) and bool((q.e == whole[i][1]).all()), (keep, i)
            else:
                step = (q.q[:, :264].view(torch.int8).int() - whole[i][0][:, :264].view(torch.int8).int()).abs()
                assert int(step.max()) <= 1 and bool((q.e == whole[i][1]).all()), keep
        c.a.q, c.b.q, c.s.q = saved
        assert float((m.mlp.y.float() - y.float()).abs().max()) <= 2 ** -6 * float(y.float().abs().max()), keep


def test_no_gradient_of_x():
    m = Mlp(100, 64, 96, 40, "bf16", "gelu", "e4m3", seed=2, need_d_x=False)
    m.forward().backward()
    sync()
    assert m.mlp.d_x is None
    m.check_backward()


def test_saved_checkpoints_are_used():
    import torch
    m = Mlp(80, 64, 160, 64, "bf16", "silu", "int8", seed=4)
    m.forward().backward()
    sync()
    n = layer.GatedMLP(m.mlp.x, m.mlp.w_gate, m.mlp.w_up, m.mlp.w_down, saved=(m.mlp.a, m.mlp.b))
    n.backward(m.dyd)
    sync()
    for t in ("d_x", "d_a", "d_b"):
        assert torch.equal(getattr(n, t), getattr(m.mlp, t)), t
    with pytest.raises(layer.MuonError):
        n.wgrad_items(m.dyd, layer.Q8(80, 64), m.mlp.w_gate, m.mlp.w_up, m.mlp.w_down)  # s was not kept


def test_repeated_calls_give_the_same_bits():
    import torch
    for sizes in ((300, 200, 330, 136), (1030, 1000, 2056, 520), (3, 200, 330, 136)):
        m = Mlp(*sizes, "bf16", "silu", "int8", seed=6)
        m.forward().backward()
        sync()
        want = [t.clone() for t in (m.mlp.y, m.mlp.d_x, m.mlp.d_a, m.mlp.d_b, m.mlp.s.q, m.mlp.s.e)]
        for _ in range(3):
            m.mlp.workspace.fill_(255)   # nothing is taken from an earlier call
            m.forward().backward()
            sync()
            for w, t in zip(want, (m.mlp.y, m.mlp.d_x, m.mlp.d_a, m.mlp.d_b, m.mlp.s.q, m.mlp.s.e)):
                assert torch.equal(w.view(torch.uint8), t.view(torch.uint8))


def test_zero_rows():
    m = Mlp(0, 64, 96, 40, "bf16", "silu", "int8", seed=2)
    m.forward().backward()
    sync()
    assert m.mlp.y.shape == (0, 40) and m.mlp.d_x.shape == (0, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,kind", [(4, None), (40, "int8"), (40, None)])
def test_infinities_and_nans_stay_in_their_rows(dtype, rows, kind):
    """A row with a NaN or an infinity has NaNs (or an infinity's sign of it); the other
    rows are what they are without it, also where K ends inside a tile."""
    def edit(m):
        m.x[1, 3] = np.nan
        m.x[2, 5] = np.inf
    clean, m = (Mlp(rows, 71, 100, 40, dtype, "silu", kind, seed=8, edit=e) for e in (None, edit))
    for t in (clean, m):
        t.forward()
    sync()
    got, want = f64(m.mlp.y), f64(clean.mlp.y)
    assert np.isnan(got[1]).all() and not np.isfinite(got[2]).any()
    keep = [r for r in range(rows) if r not in (1, 2)]
    assert (got[keep] == want[keep]).all()
    if kind:
        assert (m.mlp.a.e[1] == 255).all() and (m.mlp.s.e[2] == 255).all() and not (m.mlp.a.e[keep] == 255).any()
        for t in (clean, m):
            t.backward()
        sync()
        got, want = f64(m.mlp.d_x), f64(clean.mlp.d_x)
        assert np.isnan(got[1]).all() and (got[keep] == want[keep]).all()


def test_an_infinite_weight_meets_nothing_behind_the_end_of_k():
    """Columns of a tile past K hold other memory's infinities; none gets in."""
    import torch
    for dtype in ("bf16", "f32"):
        for inner in (40, 72):
            m = Mlp(70, 72, inner, 72, dtype, "silu", "int8", seed=3, ld=24, offset=8)   # NaNs between the rows
            m.forward().backward()
            sync()
            m.check_forward()
            m.check_backward()
            assert bool(torch.isfinite(m.mlp.d_x).all())


@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_differences(act):
    """d_x, and the weight gradients that wgrad_items give, against central differences
    of the oracle's forward pass in fp64. What the block gives differs from the formula
    by its 8-bit a, b, s and x: an int8 unit is at most 1/63.5 of a group's largest, which
    is about 2.2 sigma of these Gaussian groups of 32, so a rounding is off by
    2.2 / 63.5 / sqrt(12) = 1.0% of sigma. Up to three of them (a and b in act'(a) b, x in a
    weight gradient) and bf16's 0.2% are independent: below 3% of a gradient's norm. relu's
    slope jumps at 0: positive a below half a unit (0.017 sigma, 0.7% of them of all, 1.4%
    of the positive ones) count as 0, which is sqrt(1.4%) = 12% of the norm; 15%."""
    import torch
    m = Mlp(96, 40, 64, 48, "bf16", act, "int8", seed=11)
    m.forward().backward()
    x8 = layer.q8_save(m.mlp.x, layer.Q8(96, 40, "int8"))
    g = [torch.empty_like(w) for w in (m.mlp.w_gate, m.mlp.w_up, m.mlp.w_down)]
    layer.WGrad(m.mlp.wgrad_items(m.dyd, x8, *g)).run()
    sync()
    rng = np.random.default_rng(0)

    def loss(x, wg, wu, wd):
        return float((ref.mlp_forward(x, wg, wu, wd, act)[3] * m.dy).sum())
    at = [m.x, m.wg, m.wu, m.wd]
    off = 0.15 if act == "relu" else 0.03
    for i, got in enumerate([m.mlp.d_x, *g]):
        got = f64(got)
        for _ in range(4):
            # along a Gaussian direction d, <error, d> has the error's norm as its sigma; four
            # of them
            d = rng.standard_normal(at[i].shape)
            h = 1e-5
            plus, minus = list(at), list(at)
            plus[i], minus[i] = at[i] + h * d, at[i] - h * d
            want = (loss(*plus) - loss(*minus)) / (2 * h)
            assert abs((got * d).sum() - want) <= 4 * off * np.linalg.norm(got), (i, (got * d).sum(), want)


def test_a_site_a_block_the_weight_gradients_and_the_step_together():
    """norm site -> block -> weight gradients -> optimizer step, as a training step runs
    them, against the same in fp64 from the checkpoints that were kept."""
    import torch

    from matrix_optimizer_step_muon_amd import muon
    from oracle import muon_ref
    rows, width, inner = 200, 96, 160
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s, std=1.0: (std * torch.randn(*s, generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
    site = layer.NormSite(rand(rows, width), rand(rows, width), 1 + rand(width, std=0.1), w_post=1 + rand(width, std=0.1))
    ws = [rand(inner, width, std=width ** -0.5), rand(inner, width, std=width ** -0.5), rand(width, inner, std=inner ** -0.5)]
    before = [f64(w) for w in ws]
    nxt = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    mlp = layer.GatedMLP(site.h, *ws, act="silu", out=nxt)
    dy = rand(rows, width)
    g = [torch.empty_like(w) for w in ws]
    wgrad = layer.WGrad(mlp.wgrad_items(dy, site.u, *g, scale=site.w_pre))
    ms = [torch.zeros_like(w) for w in ws]
    plan = muon.Plan(list(zip(ws, g, ms)), lr=0.02)
    site.forward()
    mlp.forward()
    mlp.backward(dy)
    wgrad.run()
    site.backward(None, mlp.d_x)
    plan.step()
    sync()
    assert mlp.y is nxt
    from layer_helpers import codes
    u, a, b, s = (layer_ref.q8_decode(*codes(q), "int8") for q in (site.u, mlp.a, mlp.b, mlp.s))
    x = u * f64(site.w_pre)
    da, db = f64(mlp.d_a), f64(mlp.d_b)
    for got, want, mag in ((g[0], da.T @ x, np.abs(da).T @ np.abs(x)), (g[1], db.T @ x, np.abs(db).T @ np.abs(x)),
                           (g[2], f64(dy).T @ s, np.abs(f64(dy)).T @ np.abs(s))):
        err = (2 * rows + 40) * 2.0 ** -24 * mag
        assert (np.abs(f64(got) - want) <= HALF["bf16"] * np.abs(want) + err).all()
    # the step that the gradients make, at the bar of the step's own tests
    for w, w0, gr in zip(ws, before, g):
        want, _, _ = muon_ref.muon_step(w0, f64(gr), np.zeros_like(w0), lr=0.02, beta=0.95, eps=1e-7, coeffs=(3.4445, -4.7750, 2.0315),
                                        ns_steps=5, nesterov=True)
        assert np.linalg.norm(f64(w) - want) <= 2e-2 * np.linalg.norm(want)
    plan.close()


def test_past_4_gib():
    """s of 3 GiB in planes and checkpoints, rows behind 2^32 bytes: the last rows are right."""
    import torch
    free = torch.cuda.mem_get_info()[0]
    if free < 60 << 30:
        pytest.skip("needs 60 GiB")
    rows, width, inner = 70000, 32, 40960
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
    ws = [torch.randn(*s, generator=gen, device="cuda").mul_(s[1] ** -0.5).to(torch.bfloat16) for s in ((inner, width), (inner, width), (64, inner))]
    m = layer.GatedMLP(x, *ws, kind="int8")
    say("workspace", m.workspace.numel())
    m.forward()
    dy = torch.randn(rows, 64, generator=gen, device="cuda").to(torch.bfloat16)
    m.backward(dy)
    sync()
    tail = layer.GatedMLP(x[-100:], *ws, kind="int8")
    tail.forward()
    tail.backward(dy[-100:])
    sync()
    # other tiles sum in another order: all but the last bit of a rounding
    for t in ("y", "d_x"):
        p, q = f64(getattr(m, t)[-100:]), f64(getattr(tail, t))
        assert np.linalg.norm(p - q) <= 2e-3 * np.linalg.norm(q), t
    p, q = f64(m.d_b[-100:]), f64(tail.d_b)
    assert np.linalg.norm(p - q) <= 2e-3 * np.linalg.norm(q)

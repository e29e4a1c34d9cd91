"""The products' large tiles, whole, in pieces, and both in one launch: every element
against products in 64 bits on the device. What a case is for is asserted, so that
another choice of tiles cannot leave these paths untested.

Bounds by element are those of product_helpers. They are for the worst case, and grow
with the length of a sum; beside them every 64 x 64 block of a result is compared in
norm, where a wrong or missing stage of a sum shows: a bf16 result is rounded once or
twice (s, y), each time by 2^-8 at most and 2^-8 / sqrt(3) in the mean square at most, so
sqrt(2 / 3) 2^-8 and less than 2^-8 in all; an 8-bit sum's grid adds less than a tenth of
it. An fp32 result: product_helpers' unit T32 per term is for errors of one sign; the mean
square of K independent ones over the mean square of K terms is T32 / sqrt(3), doubled for
two products, and an activation's error of up to (1 + |a|) 2^-20 at |a| < 6 counts
fully: 2^-17."""

import math

import pytest

from layer_helpers import F32, HALF, say, tdt
from matrix_optimizer_step_muon_amd import layer
from product_helpers import GRID, T32

pytestmark = pytest.mark.gpu


def mm(a, b):
    """a b^T in 64 bits."""
    import torch
    return torch.mm(a.double(), b.double().t().contiguous())


def sum_error(mag, n, dtype):
    return mag * ((n + 8) * T32 if dtype == "bf16" else (6 * n + 8) * T32 + 2.1 * F32)


def activation(a, act):
    """act(a) and act'(a)."""
    import torch
    if act == "relu":
        return a.clamp(min=0), (a > 0).double()
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s + a * s * (1 - s)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-a / math.sqrt(2))
        return a * cdf, cdf + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (a + 0.044715 * a ** 3))
    return a * s, s + a * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * a * a)


def blocks(t):
    """Norms of the 64 x 64 blocks, from the first row and column and up to the last."""
    import torch
    m, n = t.shape[0] // 64 * 64, t.shape[1] // 64 * 64
    return torch.stack([v.reshape(m // 64, 64, n // 64, 64).square().sum((1, 3)).sqrt() for v in (t[:m, :n], t[-m:, -n:])])


def near(got, want, err, dtype, what):
    """By element within err and a rounding, by block within the norm above."""
    off = (got.double() - want).abs()
    over = off - err - HALF[dtype] * (want.abs() + err)
    assert float(over.max()) <= 0, (what, "by element", float(over.max()), divmod(int(over.argmax()), over.shape[1]))
    ratio = blocks(off) / blocks(want)
    assert float(ratio.max()) <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -17), (
        what, "block", int(ratio.argmax()), tuple(ratio.shape), float(ratio.max()))
    say(what, "norm of the worst block", f"{float(ratio.max()):.2e}")


def decoded(q):
    import torch
    return layer.q8_load(q, torch.empty(q.rows, q.cols, device="cuda")).double()


def check_saved(q, v, err, what):
    import torch
    unit = torch.exp2(q.e.double() - 127).repeat_interleave(32, 1)[:, :q.cols]
    half = unit / 2 if q.kind == "int8" else torch.maximum(2.0 ** -4 * v.abs(), unit * 2.0 ** -10)
    off = (decoded(q) - v).abs()
    over = off - 1.1 * err - half
    assert float(over.max()) <= 0, (what, float(over.max()), divmod(int(over.argmax()), q.cols))
    # roundings of either sign: the mean square of a half is a third of its square
    assert bool((blocks(off) <= blocks(half)).all()), what
    top = {"int8": 127.0, "e4m3": 448.0}[q.kind]
    most = torch.nn.functional.pad(v.abs() + err, (0, -q.cols % 32)).view(q.rows, -1, 32).amax(2)
    assert bool((top * torch.exp2(q.e.double() - 128) < most).all()), what + ": a coarser unit than needed"


def kinds(cuts):
    """Of each product: its tile, and whether tiles are whole (W), in pieces (P) or mixed (M)."""
    return " ".join(f"{c['tile']}{'W' if c['pieces'] == 1 else 'M' if c['whole'] else 'P'}" for c in cuts)


BLOCKS = [  # rows, width, inner, out, dtype, act, kind, what the products are for: a/b, y, ds, d_x
    (4100, 4360, 4368, 4360, "bf16", "silu", "int8", "256M 256M 256M 256M"),
    (4100, 1032, 2056, 2064, "bf16", "gelu", "e4m3", "256M 256W 256W 256P"),
    (3840, 1024, 2048, 4096, "bf16", "gelu_tanh", "e4m3", "256W 256W 256P 256P"),
    (4096, 128, 4096, 128, "bf16", "relu", "int8", "256W - 256W -"),
    (4096, 4096, 64, 4096, "bf16", "silu", "int8", "- 256W - 256W"),
    (4090, 2048, 6141, 2045, "bf16", "silu", "e4m3", "256W 256P 256W 256P"),   # operands rewritten
    (3840, 1024, 2048, 4096, "bf16", "silu", None, "256W 256W"),
    (1024, 2048, 6144, 2048, "f32", "silu", "int8", "256W 256P 256P 256P"),
    (4096, 4096, 64, 4096, "f32", "gelu", "int8", "- 256W - 256W"),
    (2200, 1040, 4360, 1032, "f32", "gelu_tanh", "e4m3", "256M 256P 256W 256P"),
    (4100, 4360, 4368, 4360, "f32", "relu", "int8", "256M 256M 256M 256M"),
]


@pytest.mark.parametrize("rows,width,inner,out,dtype,act,kind,paths", BLOCKS)
def test_blocks(rows, width, inner, out, dtype, act, kind, paths):
    import torch
    say(rows, width, inner, out, dtype, act, kind)
    g = torch.Generator(device="cuda").manual_seed(rows + inner)
    rand = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device="cuda")).to(tdt(dtype))  # noqa: E731
    x, wg, wu, wd = rand(rows, width), rand(inner, width, std=width ** -0.5), rand(inner, width, std=width ** -0.5), rand(out, inner, std=inner ** -0.5)
    m = layer.GatedMLP(x, wg, wu, wd, act=act, kind=kind)
    cuts = m.info()
    got = kinds(cuts["forward"] + cuts.get("backward", [])).split()
    assert all(w in ("-", g) for w, g in zip(paths.split(), got)) and len(got) == len(paths.split()), got
    m.forward()
    torch.cuda.synchronize()
    a, b = mm(x, wg), mm(x, wu)
    ea, eb = (sum_error(mm(x.abs(), w.abs()), width, dtype) for w in (wg, wu))
    f = activation(a, act)[0]
    s = f * b
    es = (1.13 * ea + (1 + a.abs()) * a.abs() * 2.0 ** -20) * (b.abs() + eb) + f.abs() * eb + F32 * s.abs()
    if kind:
        for q, v, e, name in ((m.a, a, ea, "a"), (m.b, b, eb, "b"), (m.s, s, es, "s")):
            check_saved(q, v, e, name)
    es = es + (HALF["bf16"] if dtype == "bf16" else 0.0) * (s.abs() + es)
    near(m.y, mm(s, wd), mm(es, wd.abs()) + sum_error(mm(s.abs() + es, wd.abs()), inner, dtype), dtype, "y")
    del a, b, ea, eb, f, s, es
    if not kind:
        return
    dy = rand(rows, out)
    m.backward(dy)
    torch.cuda.synchronize()
    a, b = decoded(m.a), decoded(m.b)
    down = wd.t().contiguous()
    ds, e = mm(dy, down), sum_error(mm(dy.abs(), down.abs()), out, dtype)
    f, df = activation(a, act)
    ef, edf = (1 + a.abs()) * a.abs() * 2.0 ** -20, (1 + a.abs()) ** 2 * 2.0 ** -20
    da, db, size = ds * b * df, ds * f, ds.abs() + e
    near(m.d_a, da, e * b.abs() * (df.abs() + edf) + size * b.abs() * edf + 2 * F32 * da.abs(), dtype, "d_a")
    near(m.d_b, db, e * (f.abs() + ef) + size * ef + F32 * db.abs(), dtype, "d_b")
    del a, b, ds, e, f, df, ef, edf, da, db, size
    gate, up, ga, gb = wg.t().contiguous(), wu.t().contiguous(), m.d_a.double(), m.d_b.double()
    mag = mm(ga.abs(), gate.abs()) + mm(gb.abs(), up.abs())
    near(m.d_x, mm(ga, gate) + mm(gb, up), sum_error(mag, 2 * inner, dtype), dtype, "d_x")


PRODUCTS = [  # rows, n, k, transposed, dtype, beta, y is c, row stride beyond the columns, offset, path
    (4100, 4360, 4112, False, "bf16", 0.5, False, 0, 0, "256M"),    # stored past the caches, with a c
    (4100, 4360, 4112, True, "bf16", 0.0, False, 0, 0, "256M"),
    (4100, 4360, 4112, True, "bf16", -1.0, True, 3, 1, "256M"),
    (2048, 2304, 8208, False, "bf16", 1.0, False, 0, 0, "256P"),
    (2048, 2304, 8208, True, "bf16", 0.0, False, 8, 8, "256M"),
    (3840, 4096, 2048, False, "bf16", 1.0, True, 0, 0, "256W"),     # through the caches, with a c
    (3840, 2048, 4100, True, "bf16", 0.0, False, 0, 0, "256W"),
    (4099, 4357, 4111, False, "bf16", 0.0, False, 0, 0, "256M"),
    (2000, 2000, 1000, False, "f32", 0.0, False, 0, 0, "128W"),
    (4100, 4360, 4112, True, "f32", 1.0, True, 0, 0, "128M"),
    (4100, 4360, 4112, False, "f32", 0.0, False, 5, 3, "128M"),
    (2048, 2304, 8208, False, "f32", 0.5, False, 0, 0, "128P"),
]


@pytest.mark.parametrize("rows,n,k,transposed,dtype,beta,in_place,ld,offset,path", PRODUCTS)
def test_8_bit_products(rows, n, k, transposed, dtype, beta, in_place, ld, offset, path):
    import torch
    say(rows, n, k, transposed, dtype, beta)
    inner, outer = (n, k) if transposed else (k, n)
    g = torch.Generator(device="cuda").manual_seed(rows + n + k)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x8 = layer.q8_save(rand(rows, inner), layer.Q8(rows, inner, "e4m3"))
    w8 = layer.w8_save(rand(n, k) * inner ** -0.5, layer.W8(n, k))
    buf = torch.full((offset + (rows + 1) * (outer + ld) + 64,), -77.0, dtype=tdt(dtype), device="cuda")
    y = torch.as_strided(buf, (rows, outer), (outer + ld, 1), offset + 32)
    c = rand(rows, outer).to(tdt(dtype))
    if in_place:
        y.copy_(c)
    p = layer.Linear8([(x8, w8, y, beta, None if in_place else c)], transposed=transposed)
    assert kinds(p.info()) == path, p.info()
    p.run()
    torch.cuda.synchronize()
    x, w = decoded(x8), layer.w8_load(w8, torch.empty(n, k, device="cuda")).double()
    w = w.t().contiguous() if transposed else w
    mag = mm(x.abs(), w.abs()) + abs(beta) * c.double().abs()
    err = mag * (inner + 8) * T32
    if dtype == "bf16":
        # the largest of a run of 16 products is at most the product of the runs' largest
        top = lambda t: torch.nn.functional.pad(t.abs(), (0, -inner % 16)).view(t.shape[0], -1, 16).amax(2)  # noqa: E731
        err = err + GRID * mm(top(x), top(w))
    near(y, mm(x, w) + beta * c.double(), err, dtype, "y")
    y.fill_(-77.0)
    assert bool((buf == -77).all()), "written around y"


def test_infos_of_several_items_and_of_few_rows():
    """The items of a call share a launch's tiles; those of few rows take none."""
    import torch
    y = lambda r, n, t=torch.bfloat16: torch.empty(r, n, dtype=t, device="cuda")  # noqa: E731
    w8 = layer.w8_save(torch.randn(300, 200, device="cuda"), layer.W8(300, 200))
    x8 = [layer.Q8(r, 200, "e4m3") for r in (0, 16, 17, 200)]
    cuts = layer.Linear8([(x, w8, y(x.rows, 300)) for x in x8]).info()
    assert [c["tile"] > 0 for c in cuts] == [False, False, True, True] and cuts[2]["tile"] == cuts[3]["tile"]
    cuts = layer.Linear8([(x, w8, y(x.rows, 300, torch.float32)) for x in x8]).info()
    assert [c["tile"] > 0 for c in cuts] == [False, True, True, True]
    rand = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    m = layer.GatedMLP(rand(1, 2048), rand(6144, 2048), rand(6144, 2048), rand(2048, 6144), kind=None)
    assert [c["tile"] for c in m.info()["forward"]] == [0, 0] and "backward" not in m.info()

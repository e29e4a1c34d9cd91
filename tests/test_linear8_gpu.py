"""8-bit weights and the 8-bit linear product against the fp64 oracle: codes bit for
bit, products within the bounds of product_helpers."""

import numpy as np
import pytest

from layer_helpers import HALF, dev, device_q8, f64, rng, say, stored, tdt, within
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref, product_ref as ref
from product_helpers import T32, grid_error

pytestmark = pytest.mark.gpu

BLOCKS = [(1, 1), (1, 300), (300, 1), (128, 128), (127, 129), (129, 127), (16, 16), (40, 1000), (257, 384), (513, 260)]


def sync():
    import torch
    torch.cuda.synchronize()


def w8_codes(w8):
    return w8.q[:, :w8.k].cpu().numpy(), None if w8.qt is None else w8.qt[:, :w8.n].cpu().numpy(), w8.e.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", BLOCKS)
def test_weight_codes(n, k, dtype):
    g = rng(n + k)
    # every block its own size, elements over the whole range of e4m3 and below it
    w = g.standard_normal((n, k)) * np.exp(3 * g.standard_normal((n, k)))
    w *= np.repeat(np.repeat(2.0 ** g.integers(-100, 100, (-(-n // 128), -(-k // 128))).astype(float), 128, 0)[:n], 128, 1)[:, :k]
    w = stored(w, dtype)
    say(n, k, dtype)
    for ld, offset in ((None, 0), (k + 3, 1)):
        w8 = layer.w8_save(dev(w, dtype, ld=ld, offset=offset), layer.W8(n, k))
        back = layer.w8_load(w8, dev(np.zeros((n, k)), dtype, ld=ld, offset=offset))
        sync()
        q, qt, e = w8_codes(w8)
        wq, we = ref.w8_encode(w)
        assert np.array_equal(e, we) and np.array_equal(q, wq) and np.array_equal(qt, wq.T)
        assert np.array_equal(f64(back), ref.w8_decode(wq, we))
    one = layer.w8_save(dev(w, dtype), layer.W8(n, k, transposed=False))
    sync()
    assert one.qt is None and np.array_equal(one.q[:, :k].cpu().numpy(), wq)


def test_weight_blocks_at_the_ends_of_the_range():
    w = np.zeros((256, 384))
    w[:128, :128] = 0.0                                       # zeros: the smallest exponent
    w[:128, 128:256] = 448.0 * 2.0 ** 20                      # exactly the top
    w[0, 128] = np.float32(448.0 * 2.0 ** 20) * (1 + 2.0 ** -20)  # just above it (fp32)
    w[:128, 256:] = 2.0 ** -126                               # below the smallest exponent's grid
    w[128:, :128] = 3.4e38
    w[130, 130] = np.inf
    w[140, 300] = np.nan
    w[200, 383] = -np.inf
    t = dev(w, "f32")
    w8 = layer.w8_save(t, layer.W8(256, 384))
    out = layer.w8_load(w8, dev(np.zeros((256, 384)), "f32"))
    sync()
    q, qt, e = w8_codes(w8)
    wq, we = ref.w8_encode(stored(w, "f32"))
    assert np.array_equal(e, we) and np.array_equal(q, wq) and np.array_equal(qt, wq.T)
    assert e[1, 1] == 255 and e[1, 2] == 255 and e[0, 0] == 17
    want = ref.w8_decode(wq, we)
    got = f64(out)
    with np.errstate(over="ignore"):
        big = np.abs(want) >= 2.0 ** 128
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isinf(got[big]).all()
    fine = ~np.isnan(want) & ~big
    assert np.array_equal(got[fine], want[fine])


class Item:
    """One product: random codes, or a saved matrix, as operands."""

    def __init__(self, rows, n, k, dtype, *, transposed=False, beta=0.0, own_c=True, seed=0, ld=0, offset=0, edit=None, w8=None,
                 spread=3):
        import torch
        g = rng(seed + rows + 3 * n + 7 * k)
        inner, outer = (n, k) if transposed else (k, n)
        self.dtype, self.beta, self.transposed = dtype, beta, transposed
        # values from 1/8 of a group's top down to subnormal codes, exponents spread over 2^+-spread
        x = g.standard_normal((rows, inner)) * np.exp(g.standard_normal((rows, inner)))
        self.q, self.e = layer_ref.q8_encode(x, "e4m3")
        self.e = np.clip(self.e.astype(int) + g.integers(-spread, spread + 1, self.e.shape), 17, 254).astype(np.uint8)
        w = g.standard_normal((n, k)) * np.exp(0.5 * g.standard_normal((n, k))) * inner ** -0.5
        self.wq, self.we = ref.w8_encode(w)
        if edit:
            edit(self)
        self.x8 = device_q8(self.q, self.e, "e4m3")
        if w8 is None:
            w8 = layer.W8(n, k)
            for t in w8.tensors():
                t.fill_(0xFF)                                   # the padding holds NaN codes
            w8.q[:, :k] = torch.from_numpy(self.wq).cuda()
            w8.qt[:, :n] = torch.from_numpy(np.ascontiguousarray(self.wq.T)).cuda()
            w8.e.copy_(torch.from_numpy(self.we))
        self.w8 = w8
        self.c = stored(2 * g.standard_normal((rows, outer)), dtype)
        self.buf = torch.full((offset + (rows + 2) * (outer + ld) + 64,), -77.0, dtype=tdt(dtype), device="cuda")
        self.y = torch.as_strided(self.buf, (rows, outer), (outer + ld, 1), offset + 32)
        C = dev(self.c, dtype)
        if beta and not own_c:
            self.y.copy_(C)
            C = None
        self.item = (self.x8, self.w8, self.y, beta, C)

    def check(self, what=""):
        x, w = layer_ref.q8_decode(self.q, self.e, "e4m3"), ref.w8_decode(self.wq, self.we)
        w = w if not self.transposed else w.T                   # outer x inner
        with np.errstate(invalid="ignore"):
            want = ref.linear(x, w, self.beta, self.c)
            mag = np.abs(x) @ np.abs(w).T + abs(self.beta) * np.abs(self.c)
            err = mag * (x.shape[1] + 8) * T32
            if self.dtype == "bf16":
                err = err + grid_error(x, w)
        within(f64(self.y), want, err + HALF[self.dtype] * (np.abs(want) + err), "y " + what)
        self.y.fill_(-77.0)
        assert bool((self.buf == -77).all()), "written around y " + what


def run(*items):
    t = items[0].transposed
    layer.Linear8([i.item for i in items], transposed=t).run()
    sync()
    for n, i in enumerate(items):
        i.check(f"of item {n}")


SIZES = [  # rows, n, k
    (1, 1, 1), (1, 200, 136), (2, 8, 16), (16, 257, 640), (17, 64, 128), (33, 40, 1000), (63, 256, 256), (64, 64, 1024), (65, 264, 272),
    (100, 203, 137), (128, 31, 513), (129, 520, 48), (257, 256, 300), (300, 700, 1), (300, 1, 700), (200, 130, 2100),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_sizes(rows, n, k, dtype, transposed):
    say(rows, n, k, dtype, transposed)
    run(Item(rows, n, k, dtype, transposed=transposed))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 90, 700])
@pytest.mark.parametrize("beta,own_c", [(1.0, True), (1.0, False), (-0.5, True)])
def test_added_to_another(rows, beta, own_c, dtype):
    run(Item(rows, 264, 200, dtype, beta=beta, own_c=own_c))
    run(Item(rows, 264, 200, dtype, transposed=True, beta=beta, own_c=own_c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,ld,offset", [(5, 8, 0), (70, 3, 1), (300, 0, 3), (300, 8, 8)])
def test_strides_and_alignments(rows, ld, offset, dtype):
    run(Item(rows, 136, 160, dtype, ld=ld, offset=offset, beta=1.0))


def test_large_tiles_whole_and_in_pieces():
    import torch
    for rows, n, k in ((2048, 2304, 1040), (1100, 1030, 2064), (4096, 4400, 128)):
        say(rows, n, k)
        g = torch.Generator(device="cuda").manual_seed(rows)
        x8 = layer.q8_save(torch.randn(rows, k, generator=g, device="cuda"), layer.Q8(rows, k, "e4m3"))
        w8 = layer.w8_save(torch.randn(n, k, generator=g, device="cuda"), layer.W8(n, k))
        y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        layer.Linear8([(x8, w8, y)]).run()
        x, w = torch.empty(rows, k, device="cuda"), torch.empty(n, k, device="cuda")
        layer.q8_load(x8, x)
        layer.w8_load(w8, w)
        x, w = x.double(), w.double()
        want = torch.mm(x, w.t().contiguous())
        mag = torch.mm(x.abs(), w.abs().t().contiguous())
        # the bound of the grid, by rows and columns: the largest of a run of 16 products is
        # at most the product of the runs' largest
        xr = torch.nn.functional.pad(x.abs(), (0, -k % 16)).view(rows, -1, 16).amax(2)
        wr = torch.nn.functional.pad(w.abs(), (0, -k % 16)).view(n, -1, 16).amax(2)
        err = 15 * 2.0 ** -13 * torch.mm(xr, wr.t().contiguous()) + mag * (k + 8) * T32
        over = (y.double() - want).abs() - err - HALF["bf16"] * (want.abs() + err)
        assert float(over.max()) <= 0, float(over.max())
        # and most of that bound is not used: the grid's errors are of either sign
        assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -8


def test_many_items_of_all_sizes():
    sizes = [(1, 40, 72), (0, 16, 32), (300, 40, 72), (64, 300, 130), (16, 7, 5), (17, 7, 5), (129, 260, 260)] * 3
    for transposed in (False, True):
        run(*[Item(r, n, k, "bf16", seed=i, transposed=transposed) for i, (r, n, k) in enumerate(sizes)])
    run(*[Item(r, n, k, "f32", seed=i) for i, (r, n, k) in enumerate(sizes)])


def test_one_weight_and_one_input_in_several_items():
    a = Item(200, 264, 136, "bf16", seed=1)
    b = Item(200, 264, 136, "bf16", seed=1, w8=a.w8)
    b.item = (a.x8,) + b.item[1:]
    run(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 80, 600])
@pytest.mark.parametrize("k", [128, 200, 4100])
def test_groups_and_blocks_of_nans(rows, k, dtype):
    """A group of x that stands for NaNs makes its row NaN, a block of w its columns;
    nothing else changes, and no NaN code of the padding counts."""
    def edit(t):
        t.e[1, -1] = 255
        t.q[1, -(k % 32 or 32):] = 0
        t.we[1, 0] = 255
        t.wq[128:256, :128] = 0
    plain, it = Item(rows, 300, k, dtype, seed=2), Item(rows, 300, k, dtype, seed=2, edit=edit)
    layer.Linear8([plain.item]).run()
    layer.Linear8([it.item]).run()
    sync()
    got, want = f64(it.y), f64(plain.y)
    assert np.isnan(got[1]).all() and np.isnan(got[:, 128:256]).all()
    keep = np.delete(np.arange(rows), 1)
    other = np.r_[0:128, 256:300]
    assert np.array_equal(got[np.ix_(keep, other)], want[np.ix_(keep, other)])


def test_extreme_exponents():
    """Scales far apart within a row: what is large decides, exactly where the sum is."""
    def edit(t):
        t.e[:] = 60
        t.e[:, 1] = 190
    run(Item(70, 130, 200, "bf16", edit=edit))
    run(Item(70, 130, 200, "f32", edit=edit))
    run(Item(9, 130, 200, "bf16", edit=edit))


def test_repeated_calls_give_the_same_bits():
    import torch
    for rows, n, k, dtype in ((300, 520, 1030, "bf16"), (1100, 1030, 2064, "bf16"), (200, 300, 2100, "f32"), (9, 300, 2100, "bf16")):
        it = Item(rows, n, k, dtype, seed=3)
        p = layer.Linear8([it.item])
        p.run()
        sync()
        want = it.y.clone()
        for _ in range(3):
            p.workspace.fill_(255)
            it.y.zero_()
            p.run()
            sync()
            assert torch.equal(it.y, want)


def test_a_linear_layer_as_it_is_trained():
    """Weights saved after a step, forward from the rounded input, gradient of the input
    from the rounded gradient, weight gradient from the same checkpoint, the next step."""
    import torch

    from matrix_optimizer_step_muon_amd import muon
    rows, n, k = 160, 136, 264
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    W, X, dY = rand(n, k, std=k ** -0.5), rand(rows, k), rand(rows, n)
    w8, x8, dy8 = layer.W8(n, k), layer.Q8(rows, k, "e4m3"), layer.Q8(rows, n, "e4m3")
    y, dx, G, M = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((rows, n), (rows, k), (n, k), (n, k)))
    fwd, bwd = layer.Linear8([(x8, w8, y)]), layer.Linear8([(dy8, w8, dx)], transposed=True)
    wgrad, plan = layer.WGrad([(dY, x8, G)]), muon.Plan([(W, G, M)])
    from layer_helpers import codes
    for _ in range(2):
        layer.w8_save(W, w8)
        layer.q8_save(X, x8)
        fwd.run()
        layer.q8_save(dY, dy8)
        bwd.run()
        wgrad.run()
        sync()
        w = ref.w8_decode(*ref.w8_encode(f64(W)))
        x, d = layer_ref.q8_decode(*codes(x8), "e4m3"), layer_ref.q8_decode(*codes(dy8), "e4m3")
        assert np.array_equal(x, layer_ref.q8_decode(*layer_ref.q8_encode(f64(X), "e4m3"), "e4m3"))
        for got, want, mag, grid, terms in ((y, x @ w.T, np.abs(x) @ np.abs(w).T, grid_error(x, w), k),
                                            (dx, d @ w, np.abs(d) @ np.abs(w), grid_error(d, w.T), n)):
            err = grid + mag * (terms + 8) * T32
            within(f64(got), want, err + HALF["bf16"] * (np.abs(want) + err), "product")
        want = f64(dY).T @ x
        err = (2 * rows + 40) * 2.0 ** -24 * (np.abs(f64(dY)).T @ np.abs(x))
        within(f64(G), want, err + HALF["bf16"] * np.abs(want), "G")
        plan.step()
    sync()
    plan.close()


def test_past_4_gib():
    """y behind 2^32 bytes."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    rows, n, k = 300000, 9000, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    x8 = layer.q8_save(torch.randn(rows, k, generator=g, device="cuda").to(torch.bfloat16), layer.Q8(rows, k, "e4m3"))
    w8 = layer.w8_save(torch.randn(n, k, generator=g, device="cuda"), layer.W8(n, k))
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    layer.Linear8([(x8, w8, y)]).run()
    few = torch.empty(16, n, dtype=torch.bfloat16, device="cuda")
    layer.Linear8([(layer.Q8(16, k, "e4m3", q=x8.q[-16:], e=x8.e[-16:]), w8, few)]).run()
    sync()
    p, q = f64(y[-16:]), f64(few)
    assert np.linalg.norm(p - q) <= 2e-3 * np.linalg.norm(q)   # another order of the same sums

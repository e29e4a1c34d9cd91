"""Weight gradients from 8-bit checkpoints against the fp64 oracle.

Tolerances. The result is rounded once to its type (HALF of its value). Before
that every product of dY and a checkpoint value is exact in fp32 (bf16 dY) or
has three parts that add up to it but for 2^-24 of it (fp32 dY), and a sum of
T products rounds at most once per product (the matrix instruction's own order
is its own; 2^-23 covers truncation), plus the scale, beta and the split's
joins.
"""

import numpy as np
import pytest

from layer_helpers import F32, HALF, dev, device_q8, f64, rng, say, stored, tdt, within
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu


def checkpoint(rows, cols, kind, seed):
    """Random codes (no NaN codes) and exponents around 1: any checkpoint a save can give."""
    g = rng(seed)
    if kind == "int8":
        q = g.integers(-127, 128, (rows, cols)).astype(np.int8).view(np.uint8)
    else:
        q = g.integers(0, 127, (rows, cols)).astype(np.uint8) | (g.integers(0, 2, (rows, cols)) * 128).astype(np.uint8)
    e = g.integers(112, 126, (rows, -(-cols // 32))).astype(np.uint8)
    return q, e


class Item:
    def __init__(self, rows, n, k, dtype, gdtype, kind, *, scale=False, beta=0.0, own_c=True, seed=0, ld=None, offset=0, ldq=None,
                 edit=None):
        import torch
        g = rng(seed + 1)
        self.dy = stored(g.standard_normal((rows, n)), dtype)
        self.q, self.e = checkpoint(rows, k, kind, seed + 2)
        if edit:
            edit(self)
        self.scale = stored(1 + 0.3 * g.standard_normal(k), dtype) if scale else None
        self.c = stored(10 * g.standard_normal((n, k)), gdtype)
        self.beta, self.dtype, self.gdtype, self.kind = beta, dtype, gdtype, kind
        # G inside a larger buffer: what lies around it stays
        self.buf = torch.full((n * k + 64,), -77.0, dtype=tdt(gdtype), device="cuda")
        self.G = self.buf[32:32 + n * k].view(n, k)
        C = dev(self.c, gdtype)
        if beta and not own_c:
            self.G.copy_(C)
            C = None
        self.item = (dev(self.dy, dtype, ld=ld, offset=offset), device_q8(self.q, self.e, kind, ldq=ldq), self.G,
                     None if self.scale is None else dev(self.scale, dtype), beta, C)

    def check(self, what=""):
        x = ref.q8_decode(self.q, self.e, self.kind)
        with np.errstate(invalid="ignore"):
            want = ref.wgrad(self.dy, x, self.scale, self.beta, self.c)
            mag = ref.wgrad(np.abs(self.dy), np.abs(x), None if self.scale is None else np.abs(self.scale), abs(self.beta), np.abs(self.c))
            tol = HALF[self.gdtype] * np.abs(want) + (2 * len(self.dy) + 40) * F32 * mag
        within(f64(self.G), want, tol, "G " + what)
        assert (self.buf[:32] == -77).all() and (self.buf[-32:] == -77).all(), "written around G"


def run(*items):
    import torch
    layer.WGrad([i.item for i in items]).run()
    torch.cuda.synchronize()
    for n, i in enumerate(items):
        i.check(f"of item {n}")


SIZES = [  # rows, n, k
    (1, 1, 1), (1, 200, 136), (2, 8, 16), (63, 256, 256), (64, 256, 256), (65, 264, 272), (100, 203, 137), (128, 31, 513),
    (129, 520, 48), (257, 256, 300), (191, 1, 700), (200, 700, 1), (1000, 72, 80), (3001, 40, 264),
]


@pytest.mark.parametrize("dtype,gdtype,kind", [("bf16", "bf16", "int8"), ("bf16", "f32", "e4m3"), ("f32", "f32", "int8"),
                                               ("f32", "bf16", "e4m3")])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_one_matrix(rows, n, k, dtype, gdtype, kind):
    say("case", rows, n, k, dtype, gdtype, kind)
    run(Item(rows, n, k, dtype, gdtype, kind, scale=rows % 2 == 0, beta=0.5 if k % 2 else 0.0, seed=rows))


# Outputs of hundreds of 256 x 256 tiles take the kernel of that tile; the ones
# above mostly the one of 64 x 64.
LARGE = [  # rows, n, k, dtype, gdtype, kind, ld, offset
    (1, 4096, 4096, "bf16", "bf16", "int8", None, 0), (63, 4104, 2100, "bf16", "f32", "e4m3", None, 0),
    (64, 2048, 4112, "bf16", "bf16", "e4m3", 2056, 8), (65, 2101, 4099, "bf16", "bf16", "int8", None, 0),
    (130, 2100, 2200, "bf16", "f32", "int8", 2111, 3), (129, 4096, 2048, "bf16", "bf16", "int8", None, 0),
    (300, 4100, 2999, "f32", "f32", "int8", None, 0), (70, 3001, 4096, "f32", "bf16", "e4m3", 3003, 1),
    (4000, 1030, 1101, "bf16", "f32", "int8", None, 0), (4033, 1024, 1200, "bf16", "bf16", "e4m3", None, 0),
]


@pytest.mark.parametrize("rows,n,k,dtype,gdtype,kind,ld,offset", LARGE)
def test_large_tiles(rows, n, k, dtype, gdtype, kind, ld, offset):
    say("case", rows, n, k, dtype, gdtype, kind, ld, offset)
    run(Item(rows, n, k, dtype, gdtype, kind, scale=k % 2 == 0, beta=0.25 if n % 2 else 1.0, own_c=n % 2 == 1, seed=rows, ld=ld,
             offset=offset))


# Between them, outputs of some hundreds of 128 x 128 tiles and shorter sums take
# the kernel of that tile, in one piece or a few.
MEDIUM = [  # rows, n, k, dtype, gdtype, kind, ld, offset
    (300, 2048, 2048, "bf16", "bf16", "int8", None, 0), (257, 1001, 5003, "bf16", "f32", "e4m3", None, 0),
    (1000, 1024, 5120, "bf16", "bf16", "e4m3", 1040, 8), (1001, 2000, 2050, "bf16", "f32", "int8", 2003, 1),
    (65, 2560, 2500, "f32", "bf16", "int8", None, 0), (300, 2040, 2100, "f32", "f32", "e4m3", None, 0),
    (2700, 1024, 1030, "bf16", "f32", "int8", None, 0), (4097, 259, 5341, "bf16", "bf16", "int8", None, 0),
    (4095, 260, 5300, "f32", "f32", "e4m3", None, 0),
]


@pytest.mark.parametrize("rows,n,k,dtype,gdtype,kind,ld,offset", MEDIUM)
def test_medium_tiles(rows, n, k, dtype, gdtype, kind, ld, offset):
    say("case", rows, n, k, dtype, gdtype, kind, ld, offset)
    run(Item(rows, n, k, dtype, gdtype, kind, scale=k % 2 == 0, beta=0.25 if n % 2 else 1.0, own_c=n % 2 == 1, seed=rows, ld=ld,
             offset=offset))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_medium_tiles_among_others(dtype):
    sizes = [(300, 2048, 1500), (0, 40, 50), (130, 700, 900), (64, 1030, 2100), (1, 129, 127)]
    run(*[Item(r, n, k, dtype, "bf16", "int8", scale=i % 2 == 0, beta=float(i % 2), seed=30 + i)
          for i, (r, n, k) in enumerate(sizes)])


@pytest.mark.parametrize("gdtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [0, 1, 100, 900])
def test_accumulation_into_g(rows, gdtype):
    say("case", rows, gdtype)
    run(Item(rows, 136, 72, "bf16", gdtype, "int8", beta=1.0, own_c=False, scale=True, seed=4))


def test_no_rows_gives_zeros():
    run(Item(0, 70, 90, "bf16", "bf16", "int8"), Item(0, 70, 90, "bf16", "bf16", "int8", beta=2.0))
    run(Item(0, 70, 90, "f32", "f32", "e4m3"))


@pytest.mark.parametrize("ld,offset,ldq", [(136, 0, 80), (144, 8, 96), (129, 0, 80), (131, 5, 112), (128, 4, 80)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignment(ld, offset, ldq, dtype):
    say("case", ld, offset, ldq, dtype)
    run(Item(77, 128, 70, dtype, "f32", "int8", ld=ld, offset=offset, ldq=ldq, scale=True))


def test_many_matrices_of_different_sizes():
    sizes = [(40 * i % 333, 8 + 24 * i, 300 - 13 * i) for i in range(19)]
    run(*[Item(r, n, k, "bf16", "bf16", "e4m3", scale=i % 3 == 0, beta=float(i % 2), seed=i) for i, (r, n, k) in enumerate(sizes)])


def test_more_tiles_than_the_gpu_has_cus():
    run(Item(96, 4100, 5000, "bf16", "bf16", "int8", seed=8))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("rows,n,k", [(70, 24, 100), (1001, 24, 100), (70, 2048, 4100), (40, 2048, 4100)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_values_reach_their_rows_and_columns_only(rows, n, k, dtype, kind):
    say("case", rows, n, k, dtype, kind)
    # An infinity in the last token's dY, where a short last stage could meet a
    # zero; a NaN elsewhere; a group of the checkpoint that stands for NaNs.
    def edit(it):
        it.dy[rows - 1, 3], it.dy[0, 9] = np.inf, np.nan
        it.e[rows // 2, 1] = 255
        it.q[rows // 2, 32:64] = 0
        it.q[rows - 1, :] = np.where(it.q[rows - 1, :] == 0, 1, it.q[rows - 1, :])  # inf * 0 would be NaN, rightly
    run(Item(rows, n, k, dtype, "f32", kind, edit=edit))


def test_extreme_magnitudes_fp32():
    def edit(it):
        g = rng(5)
        it.dy[:] = stored(it.dy * 10.0 ** g.integers(-20, 20, it.dy.shape[1]), "f32")
        it.dy[0, 0] = np.finfo(np.float32).max / 1024
        it.e[:] = 119
    run(Item(90, 48, 64, "f32", "f32", "int8", edit=edit))


def test_bits_do_not_change_between_calls_streams_or_replays():
    import torch
    it = Item(2000, 300, 200, "bf16", "f32", "int8", scale=True, beta=1.0)   # takes the split path
    plan = layer.WGrad([it.item])
    plan.run()
    torch.cuda.synchronize()
    it.check()
    want = it.G.clone()
    side = torch.cuda.Stream()
    it.G.zero_()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(side)
    side.synchronize()
    assert torch.equal(it.G, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for _ in range(3):
        it.G.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(it.G, want)
        plan.run()
        torch.cuda.synchronize()


def test_feeds_an_optimizer_step():
    # The gradients of a two-matrix layer go straight into a plan's g.
    import torch
    from matrix_optimizer_step_muon_amd import muon
    a, b = (Item(130, n, k, "bf16", "bf16", "int8", seed=n) for n, k in ((256, 128), (136, 264)))
    W = [torch.zeros_like(i.G) for i in (a, b)]
    plan = muon.Plan([(w, i.G, torch.zeros_like(w)) for w, i in zip(W, (a, b))])
    layer.WGrad([a.item, b.item]).run()
    plan.step()
    torch.cuda.synchronize()
    a.check(), b.check()
    assert all(torch.isfinite(w).all() and w.any() for w in W)


def test_python_refusals():
    import torch
    from matrix_optimizer_step_muon_amd.muon import MuonError
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q = layer.Q8(10, 64)
    G = bf(32, 64)
    site = lambda **k: layer.NormSite(bf(10, 64), bf(10, 64), bf(64), **k)  # noqa: E731
    for call in (lambda: layer.WGrad([(bf(9, 32), q, G)]),                        # rows
                 lambda: layer.WGrad([(bf(10, 32), q, bf(32, 65))]),              # columns
                 lambda: layer.WGrad([(bf(10, 32), q, bf(64, 32).t())]),          # G not contiguous
                 lambda: layer.WGrad([(bf(32, 10).t(), q, G)]),                   # dY by columns
                 lambda: layer.WGrad([(bf(1, 32).expand(10, 32), q, G)]),         # dY with row stride 0
                 lambda: layer.WGrad([(bf(10, 32), q, G), (bf(10, 32).float(), q, G.clone())]),
                 lambda: layer.WGrad([(bf(10, 32), q, G), (bf(10, 32), layer.Q8(10, 64, "e4m3"), G.clone())]),
                 lambda: layer.WGrad([(bf(10, 32), q, G), (bf(10, 32), q, G)]),   # one G twice
                 lambda: layer.WGrad([(bf(10, 32), q, G, bf(63))]),
                 lambda: layer.WGrad([(bf(10, 32), q, G, None, 1.0, bf(32, 64).float())]),
                 lambda: layer.WGrad([(bf(10, 32).half(), q, G)]),
                 lambda: layer.q8_save(bf(10, 65), q), lambda: layer.q8_load(q, bf(64, 10).t()),
                 lambda: layer.q8_save(bf(10, 64).half(), q),
                 lambda: layer.Q8(10, 64, q=q.q[:, :48], e=q.e), lambda: layer.Q8(10, 64, q=q.q, e=q.e[:, :1]),
                 lambda: layer.Q8(10, 64, q=q.q[:9], e=q.e),
                 lambda: layer.NormSite(bf(10, 64), bf(10, 63), bf(64)), lambda: layer.NormSite(bf(10, 64), bf(10, 64).float(), bf(64)),
                 lambda: layer.NormSite(bf(10, 64), bf(10, 64), bf(63)), lambda: site(gate=bf(9, 64)), lambda: site(w_post=bf(64).float()),
                 lambda: site(kind=None).backward(None, bf(10, 64)), lambda: site(kind="int4"),
                 lambda: site().backward(None, bf(10, 63)), lambda: site().backward(bf(10, 64).float(), bf(10, 64)),
                 lambda: site(res_scale=float("nan")).forward(), lambda: site(eps=-1.0).forward()):
        with pytest.raises(MuonError):
            call()
    torch.cuda.synchronize()


def test_a_raw_stream_handle_and_memory_freed_early():
    import torch
    it = Item(500, 300, 200, "bf16", "f32", "int8", scale=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = layer.WGrad([it.item])
    torch.cuda.synchronize()
    plan.run(side.cuda_stream)
    workspace = plan.workspace.numel()
    del plan                              # its workspace may not be reused before the side stream is done
    junk = torch.full((max(workspace, 1),), 255, dtype=torch.uint8, device="cuda")
    side.synchronize()
    torch.cuda.synchronize()
    it.check()
    del junk

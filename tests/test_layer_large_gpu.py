"""Tensors of more than 2^32 bytes: an offset cut to 32 bits would land in their
first rows. Only the last rows hold anything, and they are checked against the
fp64 oracle exactly as small ones are."""

import numpy as np
import pytest

from layer_helpers import F32, HALF, codes, f64, rng, say, stored, within
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu


def filled(rows, cols, last, dtype):
    """Zeros but for the last rows."""
    import torch
    t = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    t[-len(last):] = torch.from_numpy(last).to(dtype)
    return t


def test_checkpoint_past_4_gib():
    import torch
    rows, cols = 70000, 65536
    last = stored(rng(1).standard_normal((3, cols)), "bf16")
    x = filled(rows, cols, last, torch.bfloat16)
    say("case", rows, cols, x.numel() * 2, "bytes")
    ckpt = layer.q8_save(x, layer.Q8(rows, cols))
    x.fill_(5)
    layer.q8_load(ckpt, x)
    torch.cuda.synchronize()
    q, e = ref.q8_encode(last, "int8")
    assert np.array_equal(ckpt.q[-3:].cpu().numpy(), q) and np.array_equal(ckpt.e[-3:].cpu().numpy(), e)
    assert np.array_equal(f64(x[-3:]), ref.q8_decode(q, e, "int8"))
    assert not x[:-3].any()


def test_norm_site_past_4_gib():
    import torch
    rows, cols = 70000, 32768
    g = rng(2)
    b, r, dh = (stored(g.standard_normal((2, cols)), "bf16") for _ in range(3))
    w = stored(1 + 0.1 * g.standard_normal(cols), "bf16")
    wt = torch.from_numpy(w).to(torch.bfloat16).cuda()
    say("case", rows, cols, rows * cols * 2, "bytes each")
    site = layer.NormSite(filled(rows, cols, b, torch.bfloat16), filled(rows, cols, r, torch.bfloat16), wt, w_post=wt)
    site.forward()
    site.backward(None, filled(rows, cols, dh, torch.bfloat16))
    torch.cuda.synchronize()
    y, h, _, _, ry, rb = ref.norm_forward(b, r, w, w, None, 1.0, 1.0, 1e-6)
    mag = np.abs(r) + np.abs(b) * rb[:, None] * np.abs(w)
    within(f64(site.y[-2:]), y, HALF["bf16"] * np.abs(y) + 48 * F32 * mag, "y")
    within(f64(site.h[-2:]), h, HALF["bf16"] * np.abs(h) + 48 * F32 * mag * np.abs(w) * ry[:, None], "h")
    u, v = (ref.q8_decode(c.q[-2:].cpu().numpy(), c.e[-2:].cpu().numpy(), "int8") for c in (site.u, site.v))
    ry, rb = f64(site.rstd_y[-2:]), f64(site.rstd_b[-2:])
    dr, db, dw, _, _ = ref.norm_backward(np.zeros_like(dh), dh, u, v, ry, rb, w, w, None, 1.0, 1.0)
    du = np.abs(dh * w)
    ms = ry[:, None] * (du + np.abs(u) * (du * np.abs(u)).mean(1, keepdims=True))
    mb = ms * np.abs(w)
    mb = rb[:, None] * (mb + np.abs(v) * (mb * np.abs(v)).mean(1, keepdims=True))
    within(f64(site.d_residual[-2:]), dr, HALF["bf16"] * np.abs(dr) + 48 * F32 * ms, "d_residual")
    within(f64(site.d_branch[-2:]), db, HALF["bf16"] * np.abs(db) + 96 * F32 * mb, "d_branch")
    within(f64(site.d_w_pre), dw, HALF["bf16"] * np.abs(dw) + 500 * F32 * np.abs(dh * u).sum(0), "d_w_pre")
    assert not site.y[:-2].any() and not site.d_branch[:-2].any()


@pytest.mark.parametrize("n,k", [(8192, 48), (8192, 4096)])
def test_weight_gradient_past_4_gib(n, k):
    import torch
    rows = 300000
    g = rng(3)
    dy = stored(g.standard_normal((2, n)), "bf16")
    x = g.standard_normal((2, k))
    q, e = ref.q8_encode(x, "int8")
    ckpt = layer.Q8(rows, k)
    ckpt.q.zero_()
    ckpt.e.fill_(127)
    ckpt.q[-2:, :k] = torch.from_numpy(q).cuda()
    ckpt.e[-2:] = torch.from_numpy(e).cuda()
    say("case", rows, n, k, rows * n * 2, "bytes of dY")
    G = torch.full((n, k), 9.0, device="cuda")
    layer.WGrad([(filled(rows, n, dy, torch.bfloat16), ckpt, G)]).run()
    torch.cuda.synchronize()
    xv = ref.q8_decode(q, e, "int8")
    within(f64(G), ref.wgrad(dy, xv), 8 * F32 * ref.wgrad(np.abs(dy), np.abs(xv)), "G")

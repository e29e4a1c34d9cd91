"""Shared helpers of the layer operators' tests."""

from __future__ import annotations

import numpy as np

from matrix_optimizer_step_muon_amd import layer

# Half a step of a type, relative to the value: one rounding.
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
F32 = 2.0 ** -24


def tdt(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def say(*a):
    print(*a, flush=True)


def rng(seed):
    return np.random.default_rng(seed)


def dev(a, dtype, *, ld=None, offset=0):
    """a as a device tensor; with ld or offset, a view with that row stride that
    starts `offset` elements into its buffer, whose other elements are NaN."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to(tdt(dtype))
    if ld is None and offset == 0:
        return t.cuda()
    rows, cols = a.shape
    ld = ld or cols
    buf = torch.full((offset + max(rows, 1) * ld,), float("nan"), dtype=tdt(dtype), device="cuda")
    view = torch.as_strided(buf, (rows, cols), (ld, 1), offset)
    view.copy_(t)
    return view


def f64(t):
    return t.detach().cpu().double().numpy()


def stored(a, dtype):
    """a rounded to the type, in fp64."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(tdt(dtype)).double().numpy()


def codes(ckpt):
    """(q, e) of a checkpoint on the host, without its padding."""
    return ckpt.q[:, :ckpt.cols].cpu().numpy(), ckpt.e[:, :-(-ckpt.cols // layer.GROUP)].cpu().numpy()


def device_q8(q, e, kind, *, ldq=None, lde=None, fill=0xFF):
    """Host codes as a device checkpoint; the padding is `fill` (a NaN code)."""
    import torch
    rows, cols = q.shape
    ldq = ldq or -(-cols // 16) * 16
    lde = lde or e.shape[1]
    tq = torch.full((rows, ldq), fill, dtype=torch.uint8)
    te = torch.full((rows, lde), 255, dtype=torch.uint8)
    tq[:, :cols] = torch.from_numpy(q)
    te[:, :e.shape[1]] = torch.from_numpy(e)
    return layer.Q8(rows, cols, kind, q=tq.cuda(), e=te.cuda())


def within(got, want, tol, what):
    """Every element of got is within tol (same shape, >= 0) of want; where want
    is not finite, got is the same."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape, f"{what}: {got.shape} for {want.shape}"
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaNs in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities differ"
    over = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    if over.size:
        i = int(np.argmax(over))
        assert over[i] <= 0, (f"{what}: {got[fine][i]!r} for {want[fine][i]!r}, off by "
                              f"{abs(got[fine][i] - want[fine][i]):.3e}, allowed {np.broadcast_to(tol, want.shape)[fine][i]:.3e}")

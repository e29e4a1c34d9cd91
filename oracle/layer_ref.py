"""fp64 oracle of the layer operators: 8-bit checkpoints, norm sites and weight
gradients, written from their definitions in numpy. It shares no code with the
HIP path."""

from __future__ import annotations

import numpy as np

GROUP = 32
TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (sign, 4 exponent bits with bias
    7, 3 mantissa bits; no infinities, 0x7f and 0xff are NaN)."""
    t = np.empty(256)
    for c in range(128):
        e, m = c >> 3, c & 7
        t[c] = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    t[127] = np.nan
    t[128:] = -t[:128]
    return t


_E4M3 = e4m3_table()


def _nearest_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of the e4m3 numbers nearest to y (|y| <= 448), ties to the even code."""
    grid = _E4M3[:127]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def q8_encode(x: np.ndarray, kind: str):
    """(q, e) of x (rows x cols, fp64): uint8 codes and exponent bytes."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    q = np.zeros((rows, cols), np.uint8)
    e = np.zeros((rows, groups), np.uint8)
    for r in range(rows):
        for g in range(groups):
            v = x[r, g * GROUP:(g + 1) * GROUP]
            if not np.isfinite(v).all():
                e[r, g] = 255
                continue
            k = -110
            while np.abs(v).max() > TOP[kind] * 2.0 ** k:
                k += 1
            e[r, g] = k + 127
            y = v / 2.0 ** k
            code = np.rint(y).astype(np.int8).view(np.uint8) if kind == "int8" else _nearest_e4m3(y)
            q[r, g * GROUP:(g + 1) * GROUP] = code
    return q, e


def q8_decode(q: np.ndarray, e: np.ndarray, kind: str) -> np.ndarray:
    """The values that codes q (rows x cols) with exponent bytes e stand for."""
    v = q.view(np.int8).astype(np.float64) if kind == "int8" else _E4M3[q]
    unit = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return v * np.repeat(unit, GROUP, axis=1)[:, :q.shape[1]]


def norm_forward(b, r, w_pre, w_post, gate, res_scale, branch_scale, eps):
    """y, h, u, v, rstd_y, rstd_b of a norm site, all fp64 (gate: None, cols or
    rows x cols; w_post None: no norm after the block)."""
    rstd_b = np.ones(len(b)) if w_post is None else 1 / np.sqrt((b * b).mean(1) + eps)
    v = b * rstd_b[:, None]
    n = v if w_post is None else v * w_post
    n = n if gate is None else n * gate
    y = res_scale * r + branch_scale * n
    rstd_y = 1 / np.sqrt((y * y).mean(1) + eps)
    u = y * rstd_y[:, None]
    return y, u * w_pre, u, v, rstd_y, rstd_b


def norm_backward(dy, dh, u, v, rstd_y, rstd_b, w_pre, w_post, gate, res_scale, branch_scale):
    """d_residual, d_branch, d_w_pre, d_w_post, d_gate (the last two are returned
    also where the site has no such weight, as those of weights of ones)."""
    def through_norm(d, x, rstd):
        return rstd[:, None] * (d - x * (d * x).mean(1, keepdims=True))

    s = dy + through_norm(dh * w_pre, u, rstd_y)
    w2 = 1.0 if w_post is None else w_post
    gt = 1.0 if gate is None else gate
    d_gate = branch_scale * s * w2 * v
    if gate is None or gate.ndim == 1:
        d_gate = d_gate.sum(0)
    d_branch = branch_scale * s * gt * w2
    if w_post is not None:
        d_branch = through_norm(d_branch, v, rstd_b)
    return res_scale * s, d_branch, (dh * u).sum(0), (branch_scale * s * gt * v).sum(0), d_gate


def wgrad(dy, x, scale=None, beta=0.0, c=None):
    """dY^T (x * scale) + beta * c."""
    g = dy.T @ x
    g = g if scale is None else g * scale
    return g if beta == 0 else g + beta * c

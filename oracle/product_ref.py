"""fp64 oracle of the layers' products: 8-bit weights, the 8-bit linear product and
the gated feed-forward block with its backward pass, written from their
definitions in numpy. It shares no code with the HIP path."""

from __future__ import annotations

import math

import numpy as np

from .layer_ref import _nearest_e4m3, e4m3_table

BLOCK = 128
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def w8_encode(w: np.ndarray):
    """(q, e) of w (n x k, fp64): e4m3 codes, and an exponent byte per block of
    128 x 128."""
    n, k = w.shape
    q = np.zeros((n, k), np.uint8)
    e = np.zeros((-(-n // BLOCK), -(-k // BLOCK)), np.uint8)
    for i in range(e.shape[0]):
        for j in range(e.shape[1]):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            v = w[at]
            if not np.isfinite(v).all():
                e[i, j] = 255
                continue
            top, x = np.abs(v).max(), -110
            if top > 0:
                x = max(x, math.frexp(top)[1] - 12)
            while top > 448.0 * 2.0 ** x:
                x += 1
            e[i, j] = x + 127
            q[at] = _nearest_e4m3(v / 2.0 ** x)
    return q, e


def w8_decode(q: np.ndarray, e: np.ndarray) -> np.ndarray:
    n, k = q.shape
    unit = np.where(e == 255, np.nan, 2.0 ** (e.astype(float) - 127))
    return e4m3_table()[q] * np.repeat(np.repeat(unit, BLOCK, 0)[:n], BLOCK, 1)[:, :k]


def linear(x: np.ndarray, w: np.ndarray, beta: float = 0.0, c=None, transposed: bool = False) -> np.ndarray:
    with np.errstate(invalid="ignore", over="ignore"):
        y = x @ (w if transposed else w.T)
        return y + beta * c if beta else y


def activation(a: np.ndarray, act: str):
    """act(a) and act'(a)."""
    if act == "relu":
        return np.maximum(a, 0.0), (a > 0).astype(float)
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "silu":
            s = 1 / (1 + np.exp(-a))
            return a * s, s + a * s * (1 - s)
        if act == "gelu":
            cdf = 0.5 * np.vectorize(math.erfc, otypes=[float])(-a / math.sqrt(2))
            return a * cdf, cdf + a * np.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (a + 0.044715 * a ** 3))
        return a * (1 + t) / 2, (1 + t) / 2 + a / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * a * a)


def mlp_forward(x, w_gate, w_up, w_down, act):
    """(a, b, s, y)."""
    a, b = x @ w_gate.T, x @ w_up.T
    s = activation(a, act)[0] * b
    return a, b, s, s @ w_down.T


def mlp_backward(dy, a, b, w_gate, w_up, w_down, act):
    """(ds, d_a, d_b, d_x)."""
    ds = dy @ w_down
    f, df = activation(a, act)
    d_a, d_b = ds * b * df, ds * f
    return ds, d_a, d_b, d_a @ w_gate + d_b @ w_up

"""The bound that the fp32 block's results are held to in norm, on the CPU: fp32
products made of six products of bf16 parts keep it, and leaving any of the six out does
not."""

import numpy as np
import pytest

PRODUCTS = [(0, 2), (2, 0), (1, 1), (1, 2), (2, 1), (2, 2)]  # parts 0 lo, 1 mid, 2 hi

# In norm, relative, of a result of one or two sums of up to 2048 terms. A sum is made by
# 6 K / 16 instructions, each of which rounds it once: sqrt(768) roundings of 2^-24 at most
# and 2^-24 / sqrt(3) in the mean square, 9.5e-7 of the whole sum; two products in a row
# have sqrt(2) of that, 1.4e-6. What the three products left out would add is 2^-24 or so.
NORM = 2e-6


def parts(x):
    """lo, mid and hi of fp32 numbers, each the rest cut to the upper 16 bits."""
    out, rest = [], x.astype(np.float32)
    for _ in range(3):
        p = (rest.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.insert(0, p.astype(float))
        rest = rest - p
    return out


def off(k, products, seed=0):
    g = np.random.default_rng(seed + k)
    x, w = (g.standard_normal((n, k)).astype(np.float32) for n in (24, 80))
    px, pw = parts(x), parts(w)
    want = x.astype(float) @ w.astype(float).T
    got = sum(px[i] @ pw[j].T for i, j in products)
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("k", [500, 1000, 2048])
def test_all_six_products_are_needed(k):
    assert off(k, PRODUCTS) < NORM / 10
    for left_out in PRODUCTS:
        assert off(k, [p for p in PRODUCTS if p != left_out]) > 2 * NORM, left_out


def test_parts_add_up():
    x = np.random.default_rng(1).standard_normal((64, 64)).astype(np.float32)
    assert np.array_equal(sum(parts(x)), x.astype(float))

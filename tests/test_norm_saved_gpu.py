"""The norms that a site's forward pass keeps in the buffers it is given."""

import numpy as np
import pytest

from layer_helpers import F32, dev, f64, rng, say, stored, within
from matrix_optimizer_step_muon_amd import layer
from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu
DEPTH = 48  # fp32 roundings of a row's mean, its root and reciprocal, as in test_norm_site_gpu.py


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3, 33), (1000, 40), (700, 2048), (5, 5121), (300, 16384), (2, 32768)])
def test_the_branch_norm_is_written_without_a_norm_after_the_block(rows, cols, dtype):
    import torch
    say("case", rows, cols, dtype)
    g = rng(rows + cols)
    b, r = (stored(g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1))), dtype) for _ in range(2))
    w = stored(1 + 0.3 * g.standard_normal(cols), dtype)
    rstd_y, rstd_b = (torch.full((rows,), -7.0, device="cuda") for _ in range(2))
    make = lambda **k: layer.NormSite(dev(b, dtype), dev(r, dtype), dev(w, dtype), **k)  # noqa: E731
    site = make(saved=(layer.Q8(rows, cols), None, rstd_y, rstd_b))
    site.forward()
    plain = make(kind=None)
    plain.forward()
    torch.cuda.synchronize()
    want = 1 / np.sqrt((b * b).mean(1) + 1e-6)
    within(f64(rstd_b), want, DEPTH * F32 * want, "rstd_b")
    want = ref.norm_forward(b, r, w, None, None, 1.0, 1.0, 1e-6)[4]
    # a mean of squares of sums of two terms: each off by an ulp of the terms' magnitude
    mag = (np.square(np.abs(b) + np.abs(r)).mean(1) + 1e-6) * want ** 2
    within(f64(rstd_y), want, DEPTH * F32 * want * mag, "rstd_y")
    assert torch.equal(site.y, plain.y) and torch.equal(site.h, plain.h)

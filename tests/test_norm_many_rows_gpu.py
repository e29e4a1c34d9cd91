"""Norm sites with more rows than the launch has workgroups, so that every
workgroup takes several: the next row's loads in flight, the buffers of the
row sums used again, partial weight sums over rows, and their join. Against the
fp64 oracle, with the tolerances of test_norm_site_gpu.py: a weight gradient adds
a workgroup's rows, then every 16th partial sum and the 16 results, fewer
roundings than the rows / 256 + 96 allowed there (at most 1536 partial sums)."""

import pytest

from layer_helpers import codes, dev, f64, say
from oracle import layer_ref as ref
from test_norm_site_gpu import check_backward, check_forward, make, site_of

pytestmark = pytest.mark.gpu

# The most workgroups are 2560 (forward) and 1536 (backward) for 513 columns, 1280
# and 768 for 2048, 512 and 256 for 5120, and 256 for 8192 and more.
MANY = [  # rows, cols, post, gate, dtype, kind
    (6000, 513, True, "feature", "bf16", "int8"), (6000, 520, False, "none", "f32", "e4m3"),
    (3300, 2048, True, "token", "bf16", "e4m3"), (3300, 2047, False, "feature", "f32", "int8"),
    (1300, 5120, True, "feature", "bf16", "int8"), (1300, 5120, False, "token", "f32", "int8"),
    (1300, 5121, False, "none", "bf16", "int8"), (1300, 5121, True, "token", "f32", "e4m3"),
    (640, 8192, True, "none", "bf16", "int8"), (640, 8192, False, "feature", "f32", "e4m3"),
    (600, 8191, True, "token", "bf16", "e4m3"), (600, 16384, True, "feature", "bf16", "int8"),
    (600, 16383, False, "none", "f32", "int8"), (520, 32768, True, "feature", "bf16", "e4m3"),
]


@pytest.mark.parametrize("rows,cols,post,gate,dtype,kind", MANY)
def test_several_rows_per_workgroup(rows, cols, post, gate, dtype, kind):
    import torch
    say("case", rows, cols, post, gate, dtype, kind)
    d = make(rows, cols, dtype, post, gate, rows + cols)
    site = site_of(d, dtype, kind)
    site.y.fill_(float("nan"))
    site.h.fill_(float("nan"))
    site.forward()
    site.backward(dev(d["dy"], dtype), dev(d["dh"], dtype))
    torch.cuda.synchronize()
    check_forward(site, d, dtype, kind)
    u = ref.q8_decode(*codes(site.u), kind)
    v, rb = (None, None) if site.v is None else (ref.q8_decode(*codes(site.v), kind), None)
    if site.v is None:
        v = d["b"]  # nothing reads it: the branch enters the gradients as it is
    if post:
        rb = f64(site.rstd_b)
    check_backward(site, d, u, v, f64(site.rstd_y), rb, dtype)

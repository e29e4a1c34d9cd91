"""Buffers of objects that are dropped while a stream other than the one they
were made on still works on them: torch's allocator must not hand them out."""

import pytest

from layer_helpers import rng, say
from matrix_optimizer_step_muon_amd import layer
from test_wgrad_gpu import Item

pytestmark = pytest.mark.gpu


def keep_busy():
    """Some tens of milliseconds of work on the current stream."""
    import torch
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(40):
        torch.mm(a, a, out=torch.empty_like(a))


def test_a_plan_run_on_an_ambient_stream_and_dropped():
    import torch
    it = Item(5000, 300, 200, "bf16", "f32", "int8", scale=True)
    plan = layer.WGrad([it.item])
    address, size = plan.workspace.data_ptr(), plan.workspace.numel()
    say("workspace", size)
    assert size > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        keep_busy()
        plan.run()
    del plan
    junk = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert junk.data_ptr() != address
    torch.cuda.synchronize()
    it.check()


def test_gradients_made_on_one_stream_used_on_another_and_dropped():
    import torch
    x = torch.from_numpy(rng(1).standard_normal((3000, 512))).float().cuda()
    w, dh = torch.ones(512, device="cuda"), torch.ones(3000, 512, device="cuda")
    side = torch.cuda.Stream()
    site = layer.NormSite(x, x.clone(), w)
    site.forward()
    torch.cuda.synchronize()
    site.backward(None, dh, side)       # makes the gradients' memory, on side
    torch.cuda.synchronize()
    want = site.d_branch.clone()
    size = site.d_residual.numel()
    addresses = {t.data_ptr() for t in (site.d_residual, site.d_branch)}
    keep_busy()
    site.backward(None, dh)             # on the current stream
    kept = site.d_branch
    del site                            # d_residual is free, as far as side knows
    with torch.cuda.stream(side):
        junk = torch.full((size,), 5.0, device="cuda")
    assert junk.data_ptr() not in addresses
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_the_handle_of_the_default_stream_is_the_default_stream():
    import torch
    it = Item(500, 300, 200, "bf16", "f32", "int8", scale=True)
    plan = layer.WGrad([it.item])
    torch.cuda.synchronize()
    it.G.fill_(5.0)                     # on the default stream, and before the product
    plan.run(0)
    it.G.add_(0.0)                      # after it
    torch.cuda.synchronize()
    it.check()

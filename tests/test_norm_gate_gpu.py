"""Gates of a norm site by their layout: one per row, or one that all rows share."""

import pytest

from matrix_optimizer_step_muon_amd import layer
from matrix_optimizer_step_muon_amd.muon import MuonError

pytestmark = pytest.mark.gpu


def test_a_gate_whose_rows_overlap_is_refused():
    # Row stride 0 is how the C ABI spells a shared gate, whose gradient is one
    # row; a 2-D gate's gradient has a row per token.
    import torch
    x, w, g = (torch.ones(*s, device="cuda") for s in ((8, 64), (64,), (64,)))
    for gate in (g.expand(8, 64), torch.as_strided(torch.ones(128, device="cuda"), (8, 64), (1, 1))):
        with pytest.raises(MuonError, match="gate"):
            layer.NormSite(x, x.clone(), w, gate=gate)


@pytest.mark.parametrize("rows", [0, 1])
def test_a_gate_of_one_row_or_none_may_have_any_stride(rows):
    import torch
    x, w, g = (torch.ones(*s, device="cuda") for s in ((rows, 64), (64,), (64,)))
    g *= 0.25
    site = layer.NormSite(x, x.clone(), w, gate=g.expand(rows, 64))
    site.forward()
    site.backward(None, x.clone())
    torch.cuda.synchronize()
    assert site.y.shape == (rows, 64) and (site.y == 1.25).all()
    assert site.d_gate.shape == (rows, 64) and torch.isfinite(site.d_gate).all()


def test_a_wider_row_stride_stays_allowed():
    import torch
    x, w = torch.ones(8, 64, device="cuda"), torch.ones(64, device="cuda")
    gate = torch.full((8, 100), 0.5, device="cuda")[:, 10:74]
    site = layer.NormSite(x, x.clone(), w, gate=gate)
    site.forward()
    site.backward(None, x.clone())
    torch.cuda.synchronize()
    assert (site.y == 1.5).all() and torch.isfinite(site.d_gate).all()

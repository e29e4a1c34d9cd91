"""Norm sites, weight gradients and checkpoints refuse calls from another current device
than the one that their tensors are on, without a GPU."""

import pytest
import torch

from matrix_optimizer_step_muon_amd import layer
from test_layer_streams import plan, q8, site, world  # noqa: F401  (a fixture)


def test_another_current_device_is_refused(world, monkeypatch):  # noqa: F811
    (p, _), (s, _) = plan(), site()
    dh = torch.zeros(4, 64)
    s.backward(None, dh)
    world.launched.clear()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (p.run, s.forward, lambda: s.backward(None, dh), lambda: s.backward(dh, dh, 5)):
        with pytest.raises(layer.MuonError, match="cuda:0"):
            call()
    assert not world.launched


def test_checkpoints_elsewhere_are_refused(world, monkeypatch):  # noqa: F811
    def matrix(t, name, *a, **k):
        if t.data_ptr() in away:
            raise layer.MuonError(-1, f"{name} is elsewhere")
        return t
    ckpt, x, w = q8(4, 64), torch.zeros(4, 64), torch.zeros(64)
    monkeypatch.setattr(layer, "_matrix", matrix)
    away = {ckpt.q.data_ptr()}
    for call in (lambda: layer.q8_save(x, ckpt), lambda: layer.q8_load(ckpt, x),
                 lambda: layer.WGrad([(torch.zeros(4, 32), ckpt, torch.zeros(32, 64))]),
                 lambda: layer.NormSite(x, torch.zeros(4, 64), w, saved=(ckpt, None, torch.zeros(4), None))):
        with pytest.raises(layer.MuonError, match="elsewhere"):
            call()
    assert not world.launched

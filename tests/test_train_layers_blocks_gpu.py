"""The training example with gated blocks and with 8-bit weights: its gradients
against autograd of the same model in fp32, and that it runs."""

import pytest

from matrix_optimizer_step_muon_amd import layer
from test_train_layers_gpu import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def reference(model, act):
    """Loss and gradients by autograd, fp32, on copies of the model's weights; what the
    8-bit products see of them where there are such, with gradients passed straight
    through."""
    import torch
    import torch.nn.functional as F
    leaf = lambda t: None if t is None else t.float().clone().requires_grad_()  # noqa: E731
    gates, up, down = [leaf(w) for w in model.w_gate], [leaf(w) for w in model.w_up], [leaf(w) for w in model.w_down]
    for k, pair in enumerate(model.weights8):
        for w8, w in zip(pair, (up[k], down[k])):
            with torch.no_grad():
                layer.w8_load(w8, w)
    pre, post, gate = ([leaf(getattr(s, n)) for s in model.sites] for n in ("w_pre", "w_post", "gate"))
    norm = lambda x: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    f = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda v: F.gelu(v, approximate="tanh"), "relu": F.relu}
    y = model.x.float()
    h = norm(y) * pre[0]
    for k in range(len(up)):
        s = f[act](h @ gates[k].t()) * (h @ up[k].t()) if act else (h @ up[k].t()).relu().square()
        y = y + gate[k + 1] * post[k + 1] * norm(s @ down[k].t())
        h = norm(y) * pre[k + 1]
    loss = (h - model.target.float()).square().mean()
    loss.backward()
    return loss.detach(), [[w.grad for w in ws] for ws in (gates, up, down, pre)]


def compare(model, act, tol):
    import torch
    loss = model.forward()
    model.backward()
    want_loss, want = reference(model, act)
    torch.cuda.synchronize()
    assert abs(float(loss) - float(want_loss)) <= tol * float(want_loss)
    for name, gs, ws in zip(("gate", "up", "down", "w_pre"), (model.g_gate, model.g_up, model.g_down, [s.d_w_pre for s in model.sites]), want):
        assert len(gs) == len(ws)
        for k, (a, b) in enumerate(zip(gs, ws)):
            err = float((a.float() - b).norm() / b.norm())
            print(act, name, k, "relFro %.3e" % err, flush=True)
            assert err <= tol, (name, k, err)


@pytest.mark.parametrize("kind,act", [("int8", "silu"), ("e4m3", "gelu"), ("int8", "relu")])
def test_gated_gradients_against_autograd(example, kind, act):  # noqa: F811
    # Relative Frobenius error: about a dozen bf16 roundings between a loss and a
    # gradient, 2^-8 each at worst; a checkpoint value is off by half its group's
    # step at most (int8: 2^-7 of the group's top; e4m3: 2^-4 of the value, less than
    # 2^-5 on average), and up to four of them meet in one gradient: a norm's rows,
    # the two projections, and s.
    tol = 12 * 2 ** -8 + 4 * (2 ** -7 if kind == "int8" else 2 ** -5)
    if act == "relu":
        # Its derivative jumps at 0, and an a between 0 and half a unit is kept as 0,
        # whose derivative is 0. A unit is a power of two below 2 / 127 of the
        # group's top, which is 2.4 standard deviations for 32 normal numbers: of
        # the density 0.4 at 0, less than 0.4 * 2.5 / 127 of all elements, out of
        # the half that has a gradient. That share of the squares is lost in the
        # block's own gradient, and once more in the next block's d_x.
        tol += (2 * 2 * 0.4 * 2.5 / 127) ** 0.5
    compare(example.Model(300, 136, 2, kind, seed=3, act=act), act, tol)


def test_8_bit_gradients_against_autograd(example):  # noqa: F811
    # The weights are what both sides see. Every product rounds its other operand to
    # e4m3, by 2^-5 of it on average: four products on the way to the loss and four
    # back, and three checkpoints; bf16's dozen roundings as above.
    compare(example.Model(300, 136, 2, "e4m3", seed=3, weights8=True), None, 12 * 2 ** -8 + 11 * 2 ** -5)


@pytest.mark.parametrize("args", [["--act", "silu"], ["--act", "gelu_tanh", "--kind", "e4m3"], ["--weights8"]])
def test_it_runs(example, args):  # noqa: F811
    import math
    losses = example.main(["--steps", "3", "--tokens", "70", "--width", "72", "--layers", "2"] + args)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


def test_what_does_not_go_together_is_refused(example):  # noqa: F811
    with pytest.raises(ValueError):
        example.Model(8, 64, 1, "int8", weights8=True)
    with pytest.raises(ValueError):
        example.Model(8, 64, 1, "e4m3", act="silu", weights8=True)

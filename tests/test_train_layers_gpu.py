"""The training example: its gradients against autograd of the same model in
fp32, and a loss that goes down."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_layers", os.path.join(ROOT, "examples", "train_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model):
    """Loss and gradients by autograd, fp32, on copies of the model's weights."""
    import torch
    leaf = lambda t: None if t is None else t.float().clone().requires_grad_()  # noqa: E731
    up, down = [leaf(w) for w in model.w_up], [leaf(w) for w in model.w_down]
    pre, post, gate = ([leaf(getattr(s, n)) for s in model.sites] for n in ("w_pre", "w_post", "gate"))
    norm = lambda x: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    y = model.x.float()
    h = norm(y) * pre[0]
    for k in range(len(up)):
        s = (h @ up[k].t()).relu().square()
        y = y + gate[k + 1] * post[k + 1] * norm(s @ down[k].t())
        h = norm(y) * pre[k + 1]
    loss = (h - model.target.float()).square().mean()
    loss.backward()
    return loss.detach(), [w.grad for w in up], [w.grad for w in down], [w.grad for w in pre]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_gradients_against_autograd(example, kind):
    import torch
    model = example.Model(300, 128, 2, kind, seed=3)
    loss = model.forward()
    model.backward()
    want_loss, up, down, pre = reference(model)
    torch.cuda.synchronize()
    assert abs(float(loss) - float(want_loss)) <= 2 ** -6 * float(want_loss)
    # Relative Frobenius error. bf16: about a dozen roundings between a loss and a
    # gradient, 2^-8 each at worst, and the weights' share of them; a checkpoint
    # value is off by at most 1/2 of its group's step (int8: 2^-7 of the group's
    # top; e4m3: 2^-4 of the value), on average less than half of that, and up
    # to three checkpoints meet in one gradient.
    tol = 12 * 2 ** -8 + 3 * (2 ** -7 if kind == "int8" else 2 ** -5)
    for name, got, want in (("up", model.g_up, up), ("down", model.g_down, down), ("w_pre", [s.d_w_pre for s in model.sites], pre)):
        for k, (a, b) in enumerate(zip(got, want)):
            err = float((a.float() - b).norm() / b.norm())
            print(kind, name, k, "relFro %.3e" % err, flush=True)
            assert err <= tol, (name, k, err)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_the_loss_goes_down(example, kind):
    losses = example.main(["--steps", "12", "--tokens", "256", "--width", "128", "--layers", "2", "--kind", kind])
    assert losses[-1] < 0.7 * losses[0], losses

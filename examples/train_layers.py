"""A few residual MLP blocks trained end to end: norm sites with 8-bit
checkpoints, weight gradients from them, and the Muon step on the matrices.

    python examples/train_layers.py --steps 20 --tokens 1024 --width 512 --layers 2

Every block is h -> relu(h Wup^T)^2 Wdown^T, between norm sites: a norm after
the block, a gate, the residual sum, and the norm before the next block. What
the backward pass needs is kept in 8 bits only: each site's normalised rows u
and v, and the block's inner activation s. s serves twice, as the saved input of
Wdown and for the derivative of relu(a)^2, which is 2 sqrt(s). The data are
random and the target is a random linear map of the input, learnt by regression.
All buffers are made once; a training step then only launches kernels.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from matrix_optimizer_step_muon_amd import layer, muon  # noqa: E402

BF16 = torch.bfloat16


class Model:
    def __init__(self, tokens: int, width: int, layers: int, kind: str = "int8", seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device="cuda")).to(BF16)  # noqa: E731
        inner = 4 * width
        self.x = rand(tokens, width)
        self.target = (self.x.float() @ torch.randn(width, width, generator=g, device="cuda") * width ** -0.5).to(BF16)
        self.w_up = [rand(inner, width, std=width ** -0.5) for _ in range(layers)]
        self.w_down = [rand(width, inner, std=inner ** -0.5) for _ in range(layers)]
        new = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
        ones = lambda: torch.ones(width, dtype=BF16, device="cuda")  # noqa: E731
        # the site before the first block has no branch yet
        self.sites = [layer.NormSite(torch.zeros_like(self.x), self.x, ones(), kind=kind)]
        self.a = new(tokens, inner)
        self.saved = []
        for _ in range(layers):
            branch = new(tokens, width)
            self.saved.append(layer.Q8(tokens, inner, kind))
            self.sites.append(layer.NormSite(branch, self.sites[-1].y, ones(), w_post=ones(), gate=ones() * 0.5, kind=kind))
        self.dh, self.ds = new(tokens, width), new(tokens, inner)
        self.da = [new(tokens, inner) for _ in range(layers)]
        self.g_up = [torch.empty_like(w) for w in self.w_up]
        self.g_down = [torch.empty_like(w) for w in self.w_down]
        self.wgrad = None
        self.optimizer = muon.Plan([(w, d, torch.zeros_like(w)) for w, d in zip(self.w_up + self.w_down, self.g_up + self.g_down)])

    def forward(self):
        """The loss, as a device scalar."""
        self.sites[0].forward()
        for k, site in enumerate(self.sites[1:]):
            torch.mm(self.sites[k].h, self.w_up[k].t(), out=self.a)
            self.a.relu_().square_()
            layer.q8_save(self.a, self.saved[k])
            torch.mm(self.a, self.w_down[k].t(), out=site.branch)
            site.forward()
        self.diff = self.sites[-1].h.float() - self.target.float()
        return self.diff.square().mean()

    def backward(self):
        dy, dh = None, (self.diff * (2.0 / self.diff.numel())).to(BF16)
        for k in range(len(self.saved) - 1, -1, -1):
            site = self.sites[k + 1]
            site.backward(dy, dh)
            torch.mm(site.d_branch, self.w_down[k], out=self.ds)
            da = layer.q8_load(self.saved[k], self.da[k])   # s, in place
            da.sqrt_().mul_(2).mul_(self.ds)
            dy, dh = site.d_residual, torch.mm(da, self.w_up[k], out=self.dh)
        if self.wgrad is None:  # the sites' gradient buffers exist from their first backward pass on
            self.wgrad = layer.WGrad(
                [(da, site.u, g, site.w_pre) for da, site, g in zip(self.da, self.sites, self.g_up)]
                + [(site.d_branch, s, g) for site, s, g in zip(self.sites[1:], self.saved, self.g_down)])
        self.wgrad.run()
        self.sites[0].backward(dy, dh)   # the first norm's own weight gradient

    def step(self, norm_lr: float = 0.1):
        loss = self.forward()
        self.backward()
        self.optimizer.step()
        for site in self.sites:
            for w, d in ((site.w_pre, site.d_w_pre), (site.w_post, site.d_w_post), (site.gate, site.d_gate)):
                if w is not None:
                    w.sub_(d, alpha=norm_lr)
        return loss


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--kind", choices=sorted(layer.KINDS), default="int8")
    args = p.parse_args(argv)
    model = Model(args.tokens, args.width, args.layers, args.kind)
    kept = sum(q.nbytes() for s in model.sites for q in (s.u, s.v) if q is not None) + sum(q.nbytes() for q in model.saved)
    full = sum(2 * q.rows * q.cols for s in model.sites for q in (s.u, s.v) if q is not None) + sum(2 * q.rows * q.cols for q in model.saved)
    print(f"kept for the backward pass: {kept / 2**20:.1f} MiB (in bf16 {full / 2**20:.1f} MiB)")
    losses = [model.step() for _ in range(args.steps)]
    losses = [float(v) for v in torch.stack(losses).tolist()]
    for i in range(0, args.steps, max(1, args.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {args.steps - 1:4d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main()

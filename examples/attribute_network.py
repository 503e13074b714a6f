"""A network beside the Gaussians: per-Gaussian features decoded to colour and opacity, trained through the
rasterizer on a synthetic scene.

Every Gaussian has a learned feature vector; a small residual network (network.linear: 16-bit weights and
activations) turns it into the SH band-0 coefficients and the opacity logit that gs.rasterize renders.  The
gradients of features and network are clipped together to one global norm and update float32 parameters with
16-bit copies (network.Adam).

    python examples/attribute_network.py [--steps 200] [--float32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_gaussian_splatting_dgs_amd import gs, network, scenes  # noqa: E402


class AttributeNetwork:
    """features [n, width] -> (sh [n, 1, 3], opacity_logits [n])."""

    def __init__(self, n, width=64, dtype=torch.bfloat16, lr=2e-2, max_norm=1.0, seed=0):
        gen = torch.Generator().manual_seed(seed)
        shapes = [(n, width), (width, width), (width,), (width, width), (width,), (4, width), (4,)]
        scale = [0.5] + [0.0 if len(s) == 1 else s[1] ** -0.5 for s in shapes[1:]]
        self.masters = [(torch.randn(s, generator=gen) * k).cuda() for s, k in zip(shapes, scale)]
        if dtype == torch.float32:
            self.weights, copies = self.masters, None
        else:  # what the network computes with: the optimizer rounds the parameters into it
            self.weights = copies = [m.to(dtype) for m in self.masters]
        for w in self.weights:
            w.requires_grad_()
        self.opt = network.Adam([m.detach() for m in self.masters], lr=lr, max_norm=max_norm,
                                copies=None if copies is None else [c.detach() for c in copies])

    def __call__(self):
        f, w1, b1, w2, b2, w3, b3 = self.weights
        h = network.linear(f, w1, b1, act="silu")
        h = network.linear(h, w2, b2, residual=h, act="silu")
        out = network.linear(h, w3, b3).float()
        return out[:, :3].reshape(-1, 1, 3).contiguous(), out[:, 3].contiguous()

    def step(self):
        """Clipped Adam step on the gradients of the last backward; returns their global norm."""
        norm = self.opt.step([w.grad for w in self.weights])
        for w in self.weights:
            w.grad = None
        return norm


def train(steps=200, dtype=torch.bfloat16, log=print):
    """Trains on the tiny scene's own image; returns the losses (one host read at the end)."""
    sc = scenes.tiny()
    p = {k: torch.from_numpy(v).cuda() for k, v in sc.params().items()}
    rast = gs.Rasterizer(sc.cam, sc.n, sc.sh_degree)
    target = rast.forward(p).clone()
    net = AttributeNetwork(sc.n, dtype=dtype)
    losses, norms = [], []
    for _ in range(steps):
        sh, logits = net()
        image = gs.rasterize(rast, p["means"], p["log_scales"], p["quats"], logits, sh)
        loss = ((image - target) ** 2).mean()
        loss.backward()
        norms.append(net.step().clone())
        losses.append(loss.detach())
    losses, norms = torch.stack(losses).tolist(), torch.stack(norms).tolist()
    for i in range(0, steps, max(1, steps // 10)):
        log(f"step {i:4d}  loss {losses[i]:.6f}  gradient norm {norms[i]:.4f}")
    log(f"step {steps - 1:4d}  loss {losses[-1]:.6f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--float32", action="store_true")
    a = ap.parse_args()
    train(a.steps, torch.float32 if a.float32 else torch.bfloat16)

"""Attention between Gaussians and views, trained through the rasterizer on a synthetic scene.

Every view has a few learned tokens for its appearance and every Gaussian a learned feature vector.  A pre-norm block
lets the Gaussians read the tokens of the view that is rendered (layer norm, query and key/value projections, cross
attention with heads that share keys, output projection, dropout with the residual added); a linear layer turns the
result into the SH band-0 coefficients and the opacity logit that gs.rasterize renders.  Views have different numbers of
tokens, so all views' keys are one padded tensor with lengths.

    python examples/view_attention.py [--steps 200] [--float32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_gaussian_splatting_dgs_amd import gs, network, scenes  # noqa: E402


class ViewAttention:
    """features [n, width], tokens [views, count, width] -> (sh [n, 1, 3], opacity_logits [n]) for a view."""

    def __init__(self, n, token_counts, width=64, heads=4, kv_heads=2, dtype=torch.bfloat16, p=0.1, lr=1e-2, seed=0):
        self.heads, self.kv_heads, self.d, self.p = heads, kv_heads, width // heads, p
        gen = torch.Generator().manual_seed(seed)
        kv = 2 * kv_heads * self.d
        shapes = dict(features=(n, width), tokens=(len(token_counts), max(token_counts), width), norm_w=(width,),
                      norm_b=(width,), q_w=(width, width), q_b=(width,), kv_w=(kv, width), kv_b=(kv,),
                      out_w=(width, width), out_b=(width,), head_w=(4, width), head_b=(4,))
        scale = {k: s[1] ** -0.5 if k.endswith("_w") and len(s) == 2 else 0.0 for k, s in shapes.items()}
        scale.update(features=0.5, tokens=1.0)
        masters = [torch.randn(s, generator=gen).cuda() * scale[k] for k, s in shapes.items()]
        masters[list(shapes).index("norm_w")].fill_(1.0)
        copies = masters if dtype == torch.float32 else [m.to(dtype) for m in masters]
        self.weights = dict(zip(shapes, (c.requires_grad_() for c in copies)))
        self.opt = network.Adam([m.detach() for m in masters], lr=lr, max_norm=1.0,
                                copies=None if copies is masters else [c.detach() for c in copies])
        self.lengths = torch.tensor(token_counts, dtype=torch.int32, device="cuda")
        self.state = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")  # seed and step of the dropout

    def stages(self, view, state=None):
        """The block's intermediate results by name; state None: no dropout."""
        w = self.weights
        count, width = w["tokens"].shape[1:]
        s = dict(x=w["features"], t=w["tokens"][view])
        s["h"] = network.layer_norm(s["x"], w["norm_w"], w["norm_b"])
        s["q"] = network.linear(s["h"], w["q_w"], w["q_b"])
        s["kv"] = network.linear(s["t"], w["kv_w"], w["kv_b"])
        keys, values = s["kv"].view(1, count, 2, self.kv_heads, self.d).unbind(2)  # columns of one product, not copied
        s["a"] = network.cross_attention(s["q"].view(1, -1, self.heads, self.d), keys, values,
                                         k_lengths=self.lengths[view:view + 1])
        s["o"] = network.linear(s["a"].view(-1, width), w["out_w"], w["out_b"])
        s["y"] = network.dropout(s["o"], 0.0 if state is None else self.p, 0 if state is None else state, 0, s["x"])
        s["z"] = network.linear(s["y"], w["head_w"], w["head_b"])
        return s

    def __call__(self, view, state=None):
        z = self.stages(view, state)["z"].float()
        return z[:, :3].reshape(-1, 1, 3).contiguous(), z[:, 3].contiguous()

    def step(self):
        """Clipped Adam step on the gradients of the last backward; returns their global norm.  The next step draws
        another mask."""
        norm = self.opt.step([w.grad for w in self.weights.values()])
        for w in self.weights.values():
            w.grad = None
        self.state[1] += 1
        return norm


def train(steps=200, dtype=torch.bfloat16, log=print):
    """Trains on images of the tiny scene from four cameras, each in a light of its own; returns the losses, and the
    first step's gradients by name."""
    sc = scenes.tiny()
    p = {k: torch.from_numpy(v).cuda() for k, v in sc.params().items()}
    rasts = [gs.Rasterizer(cam, sc.n, sc.sh_degree) for cam in scenes.orbit_cameras(sc.cam, 4, (0.0, 0.0, 6.0))]
    targets = [r.forward(p) * light for r, light in zip(rasts, (1.0, 0.7, 0.5, 0.85))]
    net = ViewAttention(sc.n, (5, 3, 8, 1), dtype=dtype)
    losses, first = [], {}
    for i in range(steps):
        view = i % len(rasts)
        sh, logits = net(view, net.state)
        image = gs.rasterize(rasts[view], p["means"], p["log_scales"], p["quats"], logits, sh)
        loss = ((image - targets[view]) ** 2).mean()
        loss.backward()
        if i == 0:
            first = {k: w.grad.clone() for k, w in net.weights.items()}
        net.step()
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()
    for i in range(0, steps, max(1, steps // 10)):
        log(f"step {i:4d}  loss {losses[i]:.6f}")
    log(f"step {steps - 1:4d}  loss {losses[-1]:.6f}")
    return losses, first


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--float32", action="store_true")
    a = ap.parse_args()
    train(a.steps, torch.float32 if a.float32 else torch.bfloat16)

"""Layer norm, linear layers, cross attention and dropout run together, as a pre-norm attention block: each stage's
result and gradients against that stage's definition in 64 bits, from what the stages around it gave; in a graph; and
trained through the rasterizer by the example.  Each stage has the bounds of its operator's own tests; the sum of two
gradients of one tensor is one more rounding."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import test_gpu_attention as attention
import test_gpu_dropout as dropout
import test_gpu_layer_norm as norm
import test_gpu_linear as linear

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = [torch.float32, torch.float16, torch.bfloat16]
COUNTS = (70, 1, 33)


def example():
    spec = importlib.util.spec_from_file_location("view_attention", os.path.join(ROOT, "examples", "view_attention.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def block(n, dtype, **kw):
    net = example().ViewAttention(n, COUNTS, dtype=dtype, **kw)
    gen = torch.Generator().manual_seed(5)
    for k, w in net.weights.items():  # biases and norm weights that are not all alike
        if w.ndim == 1:
            w.detach().add_((0.3 * torch.randn(w.shape, generator=gen)).to(dtype).cuda())
    return net


def close(got, value, tol, what):
    value, tol = value.to(got.device), tol.to(got.device)
    bad = ~((got.double() - value).abs() <= tol)
    assert got.shape == value.shape and not bad.any(), (what, int(bad.sum()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,view,width,heads,kv_heads", [(1000, 0, 64, 4, 2), (1, 2, 64, 4, 4), (333, 1, 48, 3, 1),
                                                         (20, 2, 128, 2, 1)])
def test_stages(n, view, width, heads, kv_heads, dtype):
    net = block(n, dtype, width=width, heads=heads, kv_heads=kv_heads)
    w, u = net.weights, attention.HALF[dtype]
    print("block", n, view, width, heads, kv_heads, dtype, flush=True)
    s = net.stages(view, net.state)
    for k, t in s.items():
        if t.requires_grad and k != "x":
            t.retain_grad()
    dz = torch.from_numpy(np.random.default_rng(n).standard_normal((n, 4)).astype(np.float32)).cuda().to(dtype)
    s["z"].backward(dz)
    torch.cuda.synchronize()
    v = {k: t.detach() for k, t in s.items()}
    g = {k: t.grad for k, t in s.items()}

    def product(x, y, name, dy, dx):  # a linear layer, its weights' gradients, and its input's where that is all of it
        W, B = w[name + "_w"].detach(), w[name + "_b"].detach()
        _, value, tol, _ = linear.exact_fwd(x, W, B, None, "none")
        close(y, value, tol, name)
        want = linear.exact_bwd(x, W, B, dy, "none")
        for got, (value, tol), what in zip((dx, w[name + "_w"].grad, w[name + "_b"].grad), want, ("dx", "dw", "db")):
            close(got, value, tol, (name, what))

    product(v["y"], v["z"], "head", dz, g["y"])
    keep = dropout.keep_of(n, width, net.p, 0, 0)
    dropout.check(v["y"], v["o"], v["x"], keep, net.p)
    dropout.check(g["o"], g["y"], None, keep, net.p)
    product(v["a"].view(n, width), v["o"], "out", g["o"], g["a"].view(n, width))

    count, d = max(COUNTS), width // heads
    q, dout = v["q"].view(1, n, heads, d), g["a"].view(1, n, heads, d)
    k, vv = v["kv"].view(1, count, 2, kv_heads, d).unbind(2)
    dk, dv = g["kv"].view(1, count, 2, kv_heads, d).unbind(2)
    out, _, dq_, dk_, dv_ = attention.exact(q, k, vv, dout, None, None, net.lengths[view:view + 1], d ** -0.5)
    for got, (value, tol), what in zip((v["a"].view(q.shape), g["q"].view(q.shape), dk, dv), (out, dq_, dk_, dv_),
                                       ("out", "dq", "dk", "dv")):
        close(got, value, tol, what)

    product(v["h"], v["q"], "q", g["q"], g["h"])
    product(v["t"], v["kv"], "kv", g["kv"], g["t"])
    y, dx, dw, db = norm.exact(v["x"], w["norm_w"].detach(), w["norm_b"].detach(), g["h"], 1e-5)
    close(v["h"], *y, "h")
    close(w["norm_w"].grad, *dw, "norm dw")
    close(w["norm_b"].grad, *db, "norm db")
    value = dx[0] + g["y"].double()  # the norm's and the residual's
    close(w["features"].grad, value, dx[1] + u * value.abs() + u * dx[1] + norm.TINY[dtype], "features")
    assert not w["tokens"].grad[[i for i in range(len(COUNTS)) if i != view]].any()
    assert not g["t"][COUNTS[view]:].any()


def test_differences():
    """The block's gradients against differences, in float32, along one direction of each weight."""
    net = block(50, torch.float32)
    dz = torch.from_numpy(np.random.default_rng(1).standard_normal((50, 4)).astype(np.float32)).cuda()
    net.stages(0, net.state)["z"].backward(dz)
    gen = torch.Generator().manual_seed(2)
    for name, w in net.weights.items():
        step = torch.randn(w.shape, generator=gen).cuda() * w.detach().abs().mean()
        h, values = 2.0 ** -8, []
        with torch.no_grad():
            old = w.clone()
            for sign in (1, -1):
                w.copy_(old + sign * h * step)
                values.append(float((net.stages(0, net.state)["z"].double() * dz.double()).sum()))
            w.copy_(old)
        slope = (values[0] - values[1]) / (2 * h)
        terms = (w.grad.double() * step.double())
        # rounding: 200 outputs of size 1, each within 2^-20, over 2 h: 2^-20 sqrt(200) 2^7 < 0.002 typical, 0.03 at
        # worst; curvature: h^2 / 6 of a third derivative no larger than some hundred times the terms
        assert abs(slope - float(terms.sum())) <= 2e-3 * float(terms.abs().sum()) + 0.03, (name, slope, float(terms.sum()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_graph(dtype):
    """Forward and backward recorded once; replays with other features and another mask equal the eager block."""
    net = block(777, dtype)
    view, w = 0, list(net.weights.values())
    dz = torch.from_numpy(np.random.default_rng(1).standard_normal((777, 4)).astype(np.float32)).cuda().to(dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(net.stages(view, net.state)["z"], w, dz)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = net.stages(view, net.state)["z"]
        grads = torch.autograd.grad(z, w, dz)
    z = z.detach()
    masks = []
    for i in range(3):
        gen = torch.Generator().manual_seed(i)
        with torch.no_grad():
            w[0].copy_(torch.randn(w[0].shape, generator=gen))
        net.state[1] += 1
        net.lengths[view] = COUNTS[view] - 9 * i
        graph.replay()
        torch.cuda.synchronize()
        s = net.stages(view, net.state)
        want = torch.autograd.grad(s["z"], w, dz)
        assert torch.equal(z, s["z"]) and all(torch.equal(a, b) for a, b in zip(grads, want)), i
        masks.append(s["y"].detach() == s["x"].detach())
        del s, want
    assert not torch.equal(masks[0], masks[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_example(dtype):
    """Runs, and every weight has a gradient: all but the keys' bias, which moves all logits of a row alike, and those
    of tokens that no view has."""
    losses, first = example().train(8, dtype, log=lambda *a: None)
    assert np.isfinite(losses).all() and len(losses) == 8
    for name, g in first.items():
        assert torch.isfinite(g).all() and g.abs().sum() > 0, name
    assert first["tokens"][0, :5].abs().sum() > 0 and not first["tokens"][0, 5:].any() and not first["tokens"][1:].any()

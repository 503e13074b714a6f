"""The network operators together: the example's training through the rasterizer, and the training loop with its
gradients clipped."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_example_learns(dtype):
    spec = importlib.util.spec_from_file_location("attribute_network", os.path.join(ROOT, "examples", "attribute_network.py"))
    M = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(M)
    print("example", dtype, flush=True)
    losses = M.train(60, dtype, log=lambda *a: None)
    assert all(np.isfinite(losses)) and losses[-1] < 0.1 * losses[0], (losses[0], losses[-1])


def trainer(max_grad_norm):
    from differentiable_gaussian_splatting_dgs_amd import gs, scenes
    sc = scenes.tiny()
    p = {k: torch.from_numpy(v).cuda() for k, v in sc.params().items()}
    target = torch.from_numpy(np.random.default_rng(0).uniform(0, 1, (3, sc.cam.height, sc.cam.width)).astype(np.float32)).cuda()
    lr = dict(means=1e-3, log_scales=5e-3, quats=1e-3, opacity_logits=5e-2, sh_dc=2e-2, sh_rest=1e-3)
    return gs.Trainer(sc.cam, p, sc.sh_degree, target, lr, max_grad_norm=max_grad_norm)


def test_trainer_without_effect_of_the_clip():
    """With a norm that is never reached the clipped loop is the fused one: one step from the same state has the
    same arithmetic but for the 2D gradients' order of summation, which moves them by about 1e-6 of their terms
    (an Adam step of tiny gradients amplifies that to at most its own size, 2 lr)."""
    a, b = trainer(None), trainer(float("inf"))
    print("trainer", flush=True)
    a.step()
    b.step()
    assert float(b.clip[1]) == 1.0 and float(b.clip[0]) > 0
    assert torch.equal(a.count, b.count)
    torch.testing.assert_close(a.accum, b.accum, rtol=1e-4, atol=1e-6)
    for k in a.p:
        ga, gb = a.m[k].double(), b.m[k].double()
        assert float((ga - gb).norm()) <= 1e-4 * float(ga.norm()), k
        lr = a.lr.get(k, a.lr["sh_dc"])
        d = (a.p[k] - b.p[k]).abs()
        assert float(d.max()) <= 2.1 * lr and float((d > 1e-3 * lr).double().mean()) < 0.02, k
    assert float((b.p["quats"].norm(dim=1) - 1).abs().max()) < 1e-6


def test_trainer_clips():
    """The moments after one step hold the scaled gradients: the norm of m / 0.1 over all five groups is max_norm."""
    t = trainer(0.5)
    g = {k: torch.empty_like(v) for k, v in t.p.items()}
    t.step(grads=g)
    norm = np.sqrt(sum(float((v.double() ** 2).sum()) for v in g.values()))
    assert norm > 1.0 and abs(float(t.clip[0]) - norm) <= 1e-6 * norm
    coef = 0.5 / (norm + 1e-6)
    b1 = 1 - float(np.float32(0.9))
    for k in g:
        want = g[k].double() * coef * b1
        assert float((t.m[k].double() - want).norm()) <= 1e-6 * float(want.norm()) + 1e-30, k
    for _ in range(20):
        t.step()
    assert all(torch.isfinite(v).all() for v in t.p.values())


def test_trainer_refuses():
    from differentiable_gaussian_splatting_dgs_amd import gs
    with pytest.raises(gs.GsError):
        trainer(-1.0)

"""What network.Adam and network.GradClip keep from call to call: replaced tensors, other lists, graphs and streams."""
import pytest
import torch

pytestmark = pytest.mark.gpu

H = torch.float16


def make(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=gen, device="cuda")


def test_adam_follows_replaced_tensors():
    """Parameters, moments and copies replaced between steps, by entry and by data: the next step is that of an
    optimizer made with the new tensors, bit for bit, and the old tensors stay as they were."""
    from differentiable_gaussian_splatting_dgs_amd import network
    shapes = [(300, 4), (57,), (64, 33)]
    new = make()
    p = [new(*s) for s in shapes]
    copies = [None, None, p[2].to(H)]
    opt = network.Adam(p, lr=1e-2, max_norm=1.0, copies=copies, normalize_rows=(0,))
    opt.step([new(*s) for s in shapes])
    old = [p[0], opt.params[1].data, opt.exp_avg[1], opt.exp_avg_sq[2], copies[2]]
    kept = [t.clone() for t in old]
    opt.params[0] = new(*shapes[0])
    opt.params[1].data = new(*shapes[1])
    opt.exp_avg[1] = new(*shapes[1])
    opt.exp_avg_sq[2] = new(*shapes[2]).square()
    opt.copies[2] = torch.zeros(shapes[2], dtype=torch.bfloat16, device="cuda")
    other = network.Adam([t.clone() for t in opt.params], lr=1e-2, max_norm=1.0,
                         copies=[None, None, torch.zeros_like(opt.copies[2])], normalize_rows=(0,),
                         exp_avg=[t.clone() for t in opt.exp_avg], exp_avg_sq=[t.clone() for t in opt.exp_avg_sq])
    other.t = opt.t
    for _ in range(2):
        grads = [new(*s) for s in shapes]
        print("step", opt.t, flush=True)
        opt.step(grads)
        other.step(grads)
        for a, b in zip(opt.params + opt.exp_avg + opt.exp_avg_sq + opt.copies[2:],
                        other.params + other.exp_avg + other.exp_avg_sq + other.copies[2:]):
            assert torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(old, kept))

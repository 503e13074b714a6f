"""network.linear under autograd beyond a first derivative.  The kernels are replaced by their formulas, so that the
graph is looked at without a GPU."""
import pytest
import torch

from differentiable_gaussian_splatting_dgs_amd import gs, network


def formula(x, w, b, act):
    z = x @ w.t() + (0 if b is None else b)
    return z if act == "none" else torch.nn.functional.silu(z)


@pytest.fixture(autouse=True)
def formulas(monkeypatch):
    """gs.linear_fwd_into and gs.linear_bwd_into as detached torch operations: like the kernels, they leave no graph."""

    def fwd(x, w, b, r, y, act):
        with torch.no_grad():
            out = formula(x, w, b, act)
            return out if r is None else out + r

    def bwd(x, w, b, dy, dx, dw, db, workspace, act):
        with torch.enable_grad():
            leaves = [None if t is None else t.detach().requires_grad_() for t in (x, w, b)]
            out = formula(*leaves, act)
            got = torch.autograd.grad(out, [t for t in leaves if t is not None], dy.detach())
        for to, g in zip((dx, dw, db), got):
            if to is not None:
                to.copy_(g)

    monkeypatch.setattr(gs, "linear_fwd_into", fwd)
    monkeypatch.setattr(gs, "linear_bwd_into", bwd)


def leaves():
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(s, generator=gen).requires_grad_() for s in ((5, 3), (4, 3), (4,), (5, 4))]


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("squared", [False, True])
def test_second_derivative_raises(which, squared):
    """A penalty on a gradient, beside a term that keeps the loss differentiable: with a dy that depends on the inputs
    and with one that does not."""
    x, w, b, r = leaves()
    y = network.linear(x, w, b, r, act="silu")
    loss = y.square().sum() if squared else y.sum()
    g, = torch.autograd.grad(loss, (x, w, b)[which], create_graph=True)
    with pytest.raises(gs.GsError, match="differentiated once"):
        (loss + g.square().sum()).backward()


def test_first_derivative_of_a_kept_graph():
    """create_graph alone changes no gradient."""
    x, w, b, r = leaves()
    plain = torch.autograd.grad(network.linear(x, w, b, r, act="silu").square().sum(), (x, w, b, r))
    kept = torch.autograd.grad(network.linear(x, w, b, r, act="silu").square().sum(), (x, w, b, r), create_graph=True)
    want = torch.autograd.grad((formula(x, w, b, "silu") + r).square().sum(), (x, w, b, r))
    for p, k, v in zip(plain, kept, want):
        assert torch.equal(p, k)
        torch.testing.assert_close(p, v)


def test_second_derivative_of_the_residual():
    """The residual's gradient is dy itself, which has its own graph: its second derivative is the formula's."""
    x, w, b, r = leaves()
    g, = torch.autograd.grad(network.linear(x, w, b, r).pow(3).sum(), r, create_graph=True)
    gg, = torch.autograd.grad(g.sum(), r)
    torch.testing.assert_close(gg, 6 * (formula(x, w, b, "none") + r))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", range(4))
def test_forward_mode_raises(which, grad):
    """A tangent that the layer would drop raises; within a dual level a call without tangents is served."""
    t = [v.detach() for v in leaves()]
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(grad):
        y = network.linear(*t, act="silu")
        assert torch.equal(y, formula(*t[:3], "silu") + t[3])
        t[which] = torch.autograd.forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        with pytest.raises(NotImplementedError):
            network.linear(*t, act="silu")

"""Argument checks of the attention, layer norm and dropout calls, answered on the host before any device work, and
their functions under autograd beyond a first derivative, with the kernels replaced by their formulas."""
import ctypes as C

import pytest
import torch

from differentiable_gaussian_splatting_dgs_amd import gs, network

FAKE, ODD, HALF = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 1), C.c_void_p((1 << 20) + 2)  # never dereferenced


def attention(**kw):
    a = gs.GsAttention(batch=2, nq=5, nk=7, heads=4, kv_heads=2, d=16, dtype=0, scale=0.25)
    for f in ("q", "k", "v", "dout"):
        setattr(a, f + "_stride", (C.c_int64 * 3)(1000, 64, 16))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD = [(dict(batch=-1), -1), (dict(nq=-1), -1), (dict(nk=-1), -1), (dict(heads=0), -1), (dict(heads=-4), -1),
       (dict(kv_heads=0), -1), (dict(heads=5), -1), (dict(d=0), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1),
       (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
       (dict(d=257), -5), (dict(nq=(1 << 30) + 1), -5), (dict(nk=1 << 31), -5), (dict(batch=1 << 40), -5),
       (dict(nq=1 << 29, heads=16, kv_heads=1), -5), (dict(batch=9_000_000), -5), (dict(nk=1 << 30, batch=1 << 20), -5)]


@pytest.mark.parametrize("kw,code", BAD)
def test_attention_shapes(kw, code):
    lib, b, a = gs.load_library(), C.c_size_t(), attention(**kw)
    assert lib.gs_attention_fwd(C.byref(a), FAKE, FAKE, FAKE, None, None, None, FAKE, None, FAKE, 1 << 40, None) == code
    assert lib.gs_attention_bwd(C.byref(a), FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                FAKE, 1 << 40, None) == code
    for size in (lib.gs_attention_bwd_workspace_size, lib.gs_attention_fwd_workspace_size):
        assert size(C.byref(a), C.byref(b)) == code


def test_attention_pointers():
    lib = gs.load_library()

    def fwd(q=FAKE, k=FAKE, v=FAKE, mask=None, ql=None, kl=None, out=FAKE, lse=None, ws=FAKE, size=1 << 30, **kw):
        return lib.gs_attention_fwd(C.byref(attention(**kw)), q, k, v, mask, ql, kl, out, lse, ws, size, None)

    assert lib.gs_attention_fwd(None, FAKE, FAKE, FAKE, None, None, None, FAKE, None, None, 0, None) == -1
    assert fwd(ws=C.c_void_p((1 << 20) + 64)) == -2
    long = dict(nq=1, nk=100_000)  # few queries on many keys: the keys are split
    assert fwd(ws=None, **long) == -1 and fwd(size=64, **long) == -3
    for name in ("q", "k", "v", "out"):
        assert fwd(**{name: None}) == -1 and fwd(**{name: HALF}) == -2 and fwd(dtype=1, **{name: ODD}) == -2, name
    for name in ("ql", "kl", "lse"):
        assert fwd(**{name: HALF}) == -2, name
    assert fwd(batch=0) == 0 and fwd(nq=0, q=None, out=None) == 0

    def bwd(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, size=1 << 30, **kw):
        return lib.gs_attention_bwd(C.byref(attention(**kw)), q, k, v, None, None, None, out, lse, dout, dq, dk, dv, ws,
                                    size, None)

    for name in ("q", "k", "v", "out", "lse", "dout", "ws"):
        assert bwd(**{name: None}) == -1, name
    for name in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"):
        assert bwd(**{name: HALF}) == -2, name
    assert bwd(ws=C.c_void_p((1 << 20) + 64)) == -2 and bwd(size=0) == -3
    assert bwd(batch=0) == 0 and bwd(nq=0, nk=0) == 0
    b = C.c_size_t()
    assert lib.gs_attention_bwd_workspace_size(C.byref(attention()), None) == -1
    assert lib.gs_attention_fwd_workspace_size(C.byref(attention()), None) == -1
    assert lib.gs_attention_fwd_workspace_size(C.byref(attention()), C.byref(b)) == 0 and b.value == 0
    assert lib.gs_attention_bwd_workspace_size(C.byref(attention()), C.byref(b)) == 0 and b.value % 256 == 0
    assert bwd(size=b.value - 1) == -3


def test_layer_norm_checks():
    lib = gs.load_library()

    def shape(**kw):
        d = gs.GsLayerNorm(rows=4, n=8, dtype=0, ld_x=8, ld_y=8, ld_dx=8, eps=1e-5)
        for k, v in kw.items():
            setattr(d, k, v)
        return C.byref(d)

    def fwd(x=FAKE, w=FAKE, b=FAKE, y=FAKE, **kw):
        return lib.gs_layer_norm_fwd(shape(**kw), x, w, b, y, None)

    def bwd(x=FAKE, w=FAKE, dy=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, size=1 << 30, **kw):
        return lib.gs_layer_norm_bwd(shape(**kw), x, w, dy, dx, dw, db, ws, size, None)

    assert lib.gs_layer_norm_fwd(None, FAKE, None, None, FAKE, None) == -1
    for kw in (dict(rows=-1), dict(n=0), dict(n=-1), dict(dtype=3), dict(eps=-1.0), dict(eps=float("nan")), dict(ld_x=7),
               dict(ld_y=7), dict(x=None)):
        assert fwd(**kw) == -1 and bwd(**kw) == -1, kw
    assert fwd(y=None) == -1 and bwd(dy=None) == -1 and bwd(ld_dx=7) == -1 and bwd(ws=None) == -1
    for kw in (dict(rows=1 << 31), dict(n=(1 << 20) + 1, ld_x=1 << 21, ld_y=1 << 21, ld_dx=1 << 21)):
        assert fwd(**kw) == -5 and bwd(**kw) == -5
    for name in ("x", "w", "b", "y"):
        assert fwd(**{name: HALF}) == -2, name
    for name in ("x", "w", "dy", "dx", "dw", "db"):
        assert bwd(**{name: HALF}) == -2, name
    assert bwd(size=0) == -3 and bwd(ws=C.c_void_p((1 << 20) + 16)) == -2
    assert fwd(rows=0, x=None, y=None) == 0 and bwd(dx=None, dw=None, db=None) == 0
    assert lib.gs_layer_norm_bwd_workspace_size(shape(), None) == -1


def test_dropout_checks():
    lib = gs.load_library()

    def call(state=None, x=FAKE, r=None, y=FAKE, **kw):
        d = gs.GsDropoutArgs(rows=4, n=8, dtype=0, ld_x=8, ld_y=8, ld_res=8, p=0.5, seed=1, offset=0)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.gs_dropout(C.byref(d), state, x, r, y, None)

    assert lib.gs_dropout(None, None, FAKE, None, FAKE, None) == -1
    for kw in (dict(rows=-1), dict(n=-1), dict(dtype=3), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(ld_x=7),
               dict(ld_y=7), dict(r=FAKE, ld_res=7), dict(x=None), dict(y=None)):
        assert call(**kw) == -1, kw
    assert call(rows=1 << 31) == -5 and call(n=(1 << 20) + 1, ld_x=1 << 21, ld_y=1 << 21) == -5
    for name in ("x", "r", "y"):
        assert call(**{name: HALF}) == -2, name
    assert call(state=C.c_void_p((1 << 20) + 4)) == -2
    assert call(rows=0, x=None, y=None) == 0 and call(n=0) == 0


def test_python_checks():
    """Tensors that the calls refuse: not on a GPU, or of another kind."""
    q, k = torch.zeros(1, 2, 4, 8), torch.zeros(1, 3, 2, 8)
    for bad in ((q, k, k), (q[0], k, k), (q, None, k), (q.int(), k, k)):
        with pytest.raises(gs.GsError):
            network.cross_attention(*bad)
        with pytest.raises(gs.GsError):
            network.cross_attention_forward(*bad)
    x = torch.zeros(3, 4)
    for call in (lambda: network.layer_norm(x), lambda: network.layer_norm(x[0]), lambda: network.dropout(x, 0.5, 1),
                 lambda: network.layer_norm_backward(x, x), lambda: network.dropout_backward(x, 0.5, 1),
                 lambda: network.cross_attention_backward(q, q, k, k, q, x)):
        with pytest.raises(gs.GsError):
            call()


# The functions, with formulas for kernels.

def attend(q, k, v, scale):
    group = q.shape[2] // k.shape[2]
    q, k, v = q.transpose(1, 2), *(t.transpose(1, 2).repeat_interleave(group, 1) for t in (k, v))
    return torch.softmax(q @ k.transpose(2, 3) * (q.shape[3] ** -0.5 if scale is None else scale), 3) @ v


def gradients(function, tensors, outs, upstream):
    """Into outs (None: not wanted), with no graph left: what a kernel does."""
    with torch.enable_grad():
        leaves = [t.detach().requires_grad_() for t in tensors]
        got = torch.autograd.grad(function(*leaves), leaves, upstream.detach())
    for to, g in zip(outs, got):
        if to is not None:
            to.copy_(g)


@pytest.fixture
def formulas(monkeypatch):
    def attention_fwd(q, k, v, mask, ql, kl, out, lse, ws, scale):
        with torch.no_grad():
            return attend(q, k, v, scale).transpose(1, 2), torch.zeros(())

    def attention_bwd(q, k, v, out, lse, dout, dq, dk, dv, ws, mask, ql, kl, scale):
        gradients(lambda *t: attend(*t, scale).transpose(1, 2), (q, k, v), (dq, dk, dv), dout)

    def norm_fwd(x, w, b, y, eps):
        with torch.no_grad():
            return torch.nn.functional.layer_norm(x, x.shape[1:], w, b, eps)

    def norm_bwd(x, w, dy, dx, dw, db, ws, eps):
        gradients(lambda *t: torch.nn.functional.layer_norm(t[0], x.shape[1:], t[1], t[2], eps),
                  (x, w, torch.zeros_like(w)), (dx, dw, db), dy)

    def drop(x, p, seed, offset, residual, y):
        with torch.no_grad():
            keep = (torch.arange(x.numel()).view(x.shape) % 3 != 0).to(x.dtype)
            return x * keep * 1.5 + (0 if residual is None else residual)

    for name, f in (("attention_fwd_into", attention_fwd), ("attention_bwd_into", attention_bwd),
                    ("layer_norm_fwd_into", norm_fwd), ("layer_norm_bwd_into", norm_bwd), ("dropout_into", drop)):
        monkeypatch.setattr(gs, name, f)


def leaves(*shapes):
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(s, generator=gen).requires_grad_() for s in shapes]


CALLS = {"attention": (lambda *t: network.cross_attention(*t), ((2, 3, 4, 5), (2, 6, 2, 5), (2, 6, 2, 5))),
         "norm": (lambda *t: network.layer_norm(*t), ((4, 6), (6,), (6,)))}


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("call", CALLS)
def test_second_derivative_raises(formulas, call, which):
    function, shapes = CALLS[call]
    t = leaves(*shapes)
    loss = function(*t).square().sum()
    g, = torch.autograd.grad(loss, t[which], create_graph=True)
    with pytest.raises(gs.GsError, match="differentiated once"):
        (loss + g.square().sum()).backward()


@pytest.mark.parametrize("call", CALLS)
def test_first_derivative(formulas, call):
    function, shapes = CALLS[call]
    t = leaves(*shapes)
    want = {"attention": lambda: attend(*t, None).transpose(1, 2),
            "norm": lambda: torch.nn.functional.layer_norm(t[0], (6,), t[1], t[2])}[call]()
    plain = torch.autograd.grad(function(*t).square().sum(), t)
    kept = torch.autograd.grad(function(*t).square().sum(), t, create_graph=True)
    for p, k, w in zip(plain, kept, torch.autograd.grad(want.square().sum(), t)):
        assert torch.equal(p, k)
        torch.testing.assert_close(p, w)


def test_dropout_is_linear(formulas):
    """Its gradient is the same call, which is differentiable again; the residual's is dy."""
    x, r = leaves((4, 6), (4, 6))
    g, gr = torch.autograd.grad(network.dropout(x, 1 / 3, 1, residual=r).pow(3).sum(), (x, r), create_graph=True)
    gg, = torch.autograd.grad(g.sum(), x)
    keep = (torch.arange(24).view(4, 6) % 3 != 0).float() * 1.5
    torch.testing.assert_close(gg, 6 * (x * keep + r) * keep * keep)
    torch.testing.assert_close(gr, 3 * (x * keep + r) ** 2)


@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_raises(formulas, grad):
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(grad):
        for function, shapes in (*CALLS.values(), (lambda *t: network.dropout(t[0], 0.5, 1, residual=t[1]),
                                                   ((3, 4), (3, 4)))):
            t = [v.detach() for v in leaves(*shapes)]
            function(*t)
            for i in range(len(t)):
                dual = list(t)
                dual[i] = torch.autograd.forward_ad.make_dual(t[i], torch.ones_like(t[i]))
                with pytest.raises(NotImplementedError):
                    function(*dual)

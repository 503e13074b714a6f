"""Argument checks of the network calls that the host answers before any device work."""
import ctypes as C

import pytest


def lin(gs, **kw):
    d = gs.GsLinear(rows=4, n_in=8, n_out=6, dtype=0, act=2, ld_x=8, ld_y=6, ld_res=6, ld_dx=8)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


FAKE = C.c_void_p(1 << 20)  # never dereferenced: every call below fails its checks first


def test_linear_checks():
    from differentiable_gaussian_splatting_dgs_amd import gs
    lib = gs.load_library()

    def fwd(x=FAKE, w=FAKE, b=FAKE, r=FAKE, y=FAKE, **kw):
        return lib.gs_linear_fwd(C.byref(lin(gs, **kw)), x, w, b, r, y, None)

    assert lib.gs_linear_fwd(None, FAKE, FAKE, None, None, FAKE, None) == -1
    for kw in (dict(rows=-1), dict(n_in=-1), dict(n_out=-1), dict(dtype=3), dict(dtype=-1), dict(act=4), dict(act=-1),
               dict(ld_x=7), dict(ld_y=5), dict(ld_res=5), dict(ld_x=-8), dict(x=None), dict(w=None), dict(y=None)):
        assert fwd(**kw) == -1, kw
    assert fwd(rows=1 << 31) == -5 and fwd(n_in=(1 << 20) + 1, ld_x=1 << 21) == -5
    odd = C.c_void_p((1 << 20) + 2)
    for k in ("x", "w", "b", "r", "y"):
        assert fwd(**{k: odd}) == -2, k
    assert fwd(rows=0, x=None, w=None, y=None) == 0 and fwd(n_out=0, y=None) == 0

    def bwd(ws=FAKE, size=1 << 30, x=FAKE, dy=FAKE, dx=FAKE, dw=FAKE, db=FAKE, **kw):
        return lib.gs_linear_bwd(C.byref(lin(gs, **kw)), x, FAKE, FAKE, dy, dx, dw, db, ws, size, None)

    for kw in (dict(rows=-1), dict(dtype=7), dict(act=9), dict(ld_x=7), dict(ld_y=5), dict(ld_dx=7), dict(x=None),
               dict(dy=None), dict(ws=None)):
        assert bwd(**kw) == -1, kw
    assert bwd(size=0) == -3
    assert bwd(ws=C.c_void_p((1 << 20) + 16)) == -2 and bwd(dx=odd) == -2 and bwd(dw=odd) == -2
    b = C.c_size_t()
    assert lib.gs_linear_bwd_workspace_size(C.byref(lin(gs)), None) == -1
    assert lib.gs_linear_bwd_workspace_size(C.byref(lin(gs)), C.byref(b)) == 0 and b.value % 256 == 0


def test_clip_checks():
    from differentiable_gaussian_splatting_dgs_amd import gs
    lib = gs.load_library()
    t = (gs.GsGradTensor * 2)()
    for a in t:
        a.grad, a.out, a.count, a.dtype = 1 << 20, 1 << 20, 10, 0
    inf = float("inf")

    def norm(n=2, arr=t, max_norm=1.0, clip=FAKE, ws=FAKE, size=1 << 20):
        return [f(n, arr, max_norm, clip, ws, size, None) for f in (lib.gs_grad_norm, lib.gs_grad_clip)]

    for kw in (dict(n=-1), dict(arr=None), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=-inf),
               dict(clip=None), dict(ws=None)):
        assert norm(**kw) == [-1, -1], kw
    assert norm(size=8) == [-3, -3]
    assert norm(clip=C.c_void_p((1 << 20) + 4)) == [-2, -2] and norm(ws=C.c_void_p((1 << 20) + 8)) == [-2, -2]
    for field, value, code in (("dtype", 3, -1), ("count", -1, -1), ("grad", None, -1), ("grad", (1 << 20) + 2, -2),
                               ("count", 1 << 50, -5)):
        keep = getattr(t[1], field)
        setattr(t[1], field, value)
        assert norm() == [code, code], field
        setattr(t[1], field, keep)
    b = C.c_size_t()
    assert lib.gs_grad_workspace_size(-1, C.byref(b)) == -1 and lib.gs_grad_workspace_size(1, None) == -1
    assert gs.gs_grad_workspace_size(1) > 0 and gs.gs_grad_workspace_size(300) > gs.gs_grad_workspace_size(1)


def test_adam_checks():
    from differentiable_gaussian_splatting_dgs_amd import gs
    lib = gs.load_library()
    assert lib.gs_adam_step_clipped(0, None, 0.9, 0.999, 1e-8, 1, None, None) == 0

    def adam(step=1, clip=None, **kw):
        t = (gs.GsAdamTensor * 1)()
        a = t[0]
        a.param = a.grad = a.exp_avg = a.exp_avg_sq = 1 << 20
        a.rows, a.row_len, a.col_end, a.lr = 10, 4, 4, 1e-3
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.gs_adam_step_clipped(1, t, 0.9, 0.999, 1e-8, step, clip, None)

    for kw in (dict(step=0), dict(rows=-1), dict(row_len=0), dict(col_begin=-1), dict(col_end=5), dict(col_begin=4),
               dict(grad_dtype=3), dict(copy=1 << 20, copy_dtype=5), dict(param=None), dict(grad=None),
               dict(exp_avg=None), dict(exp_avg_sq=None), dict(normalize_rows=1, col_begin=1)):
        assert adam(**kw) == -1, kw
    for kw in (dict(param=(1 << 20) + 2), dict(grad=(1 << 20) + 1, grad_dtype=2), dict(copy=(1 << 20) + 1, copy_dtype=1),
               dict(clip=C.c_void_p((1 << 20) + 4))):
        assert adam(**kw) == -2, kw
    assert adam(rows=1 << 40) == -5


def test_python_checks():
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    import torch
    with pytest.raises(gs.GsError):
        network.GradClip(-1.0)
    with pytest.raises(gs.GsError):
        network.linear(torch.zeros(2, 3), torch.zeros(4, 3))  # not on a GPU

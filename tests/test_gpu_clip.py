"""Gradient clipping and the clipped Adam step on the GPU (gs_grad_norm, gs_grad_clip, gs_adam_step_clipped,
network.GradClip, network.Adam) against their definition in 64 bits.

Bounds.  The squares are summed in float64, so the norm is its float32 rounding (u = 2^-24, doubled for the
square root's and the sum's own float64 errors) and the coefficient likewise.  A clipped value is the float32 product
rounded to its type.  In the Adam step m and v are two products and a sum in float32 of factors that are each
rounded (6 u of their terms); the update uses a hardware square root and reciprocal (1 ulp each, 2 u) and five
further roundings."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
U32 = 2.0 ** -24


def grads_of(spec, seed=0, scale=0.3, lead=0):
    """CUDA gradients for a list of (shape, dtype), `lead` elements into their buffers."""
    rng = np.random.default_rng(seed)
    out = []
    for shape, dtype in spec:
        n = math.prod(shape)
        buf = torch.zeros(n + lead, dtype=dtype, device="cuda")
        buf[lead:] = torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)).to(dtype)
        out.append(buf[lead:].view(shape))
    return out


def norm64(grads):
    return math.sqrt(sum(float((g.cpu().double() ** 2).sum()) for g in grads))


F, H, B = torch.float32, torch.float16, torch.bfloat16
LISTS = {
    "one element": [((1,), F)],
    "empty among others": [((0,), F), ((5, 3), F), ((0, 4), H), ((7,), B), ((0,), B)],
    "gaussians": [((3001, 3), F), ((3001, 3), F), ((3001, 4), F), ((3001,), F), ((3001, 16, 3), F)],
    "mixed network": [((59, 64), H), ((59,), H), ((128, 63), B), ((128,), B), ((1021, 33), F), ((1021,), F)],
    "whole chunks": [((4096,), F), ((8192,), H), ((8193,), B), ((4095,), F), ((1 << 20,), F)],
    "many": [((k % 37 + 1, 3), (F, H, B)[k % 3]) for k in range(200)],
    "sixty-four": [((5,), F)] * 64,
    "long": [((30_000_001,), B), ((12_000_003,), F)],
}


@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("max_norm", [0.0, 0.7, 1e9, math.inf])
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name, max_norm, lead):
    from differentiable_gaussian_splatting_dgs_amd import network
    grads = grads_of(LISTS[name], lead=lead)
    before = [g.clone() for g in grads]
    print(name, max_norm, lead, flush=True)
    clip = network.GradClip(max_norm)
    want = norm64(grads)
    assert abs(float(clip.norm(grads)) - want) <= 2 * U32 * want
    coef = min(1.0, max_norm / (want + 1e-6))
    assert abs(float(clip.state[1]) - coef) <= 2 * U32 * coef
    out = [torch.full_like(g, 9.0) for g in grads]
    assert abs(float(clip.clip(grads, out=out)) - want) <= 2 * U32 * want
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    for g, o in zip(grads, out):
        v = g.cpu().double() * coef
        assert ((o.cpu().double() - v).abs() <= (U[g.dtype] * (1 + 4 * U32) + 4 * U32) * v.abs() + TINY[g.dtype]).all()
        if coef == 1.0:
            assert torch.equal(o, g)
    clip.clip(grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


def test_buffers_around_are_untouched():
    from differentiable_gaussian_splatting_dgs_amd import network
    for dtype in (F, H, B):
        buf = torch.ones(20_000, dtype=dtype, device="cuda")
        g = buf[101:101 + 9001]
        network.GradClip(0.5).clip([g])
        assert (buf[:101] == 1).all() and (buf[101 + 9001:] == 1).all() and (g < 0.01).all()


def test_norm_beyond_float32_squares():
    """Gradients whose squares overflow or vanish in float32."""
    from differentiable_gaussian_splatting_dgs_amd import network
    for v in (1e30, 1e-30):
        g = [torch.full((1000,), v, device="cuda"), torch.full((24,), -v, device="cuda")]
        assert abs(float(network.GradClip(1.0).norm(g)) - 32 * v) <= 1e-6 * 32 * v
    g = [torch.full((1 << 12,), 3e38, device="cuda")]  # the norm itself is past float32: the clip still works
    c = network.GradClip(64.0)
    assert math.isinf(float(c.clip(g)))
    assert abs(float(g[0][0]) - 1.0) <= 1e-4  # the coefficient is subnormal: few bits


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_norm_changes_nothing(bad):
    from differentiable_gaussian_splatting_dgs_amd import network
    for dtype in (F, H, B):
        grads = grads_of([((100, 3), F), ((5000,), dtype)])
        grads[1][4321] = bad
        before = [g.clone() for g in grads]
        c = network.GradClip(0.1)
        n = float(c.clip(grads))
        assert not math.isfinite(n) and math.isnan(float(c.state[1]))
        assert all(torch.equal(a.nan_to_num(1, 2, 3), b.nan_to_num(1, 2, 3)) for a, b in zip(grads, before))
        p = [torch.randn_like(g.float()) for g in grads]
        opt = network.Adam(p, lr=0.1, max_norm=0.1)
        kept = [t.clone() for t in p]
        opt.step(grads)
        assert all(torch.equal(a, b) for a, b in zip(p, kept))
        assert all((t == 0).all() for t in opt.exp_avg + opt.exp_avg_sq)


def test_state_survives_other_lists():
    """One GradClip over lists of different lengths and sizes, back and forth."""
    from differentiable_gaussian_splatting_dgs_amd import network
    c = network.GradClip(1.0)
    for name in ("many", "one element", "gaussians", "many", "whole chunks"):
        g = grads_of(LISTS[name], seed=3)
        assert abs(float(c.norm(g)) - norm64(g)) <= 2 * U32 * norm64(g), name


def adam64(g, p, m, v, lr, t, coef, b1=0.9, b2=0.999, eps=1e-8):
    g = coef * g
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    step = lr * (m2 / (1 - b1 ** t)) / (torch.sqrt(v2 / (1 - b2 ** t)) + eps)
    return p - step, m2, v2, step


@pytest.mark.parametrize("name", [n for n in LISTS if n != "long"])
@pytest.mark.parametrize("max_norm", [None, 0.7, 1e9])
def test_adam(name, max_norm):
    """Three steps, each compared from the state before it; 16-bit gradients keep a 16-bit copy."""
    from differentiable_gaussian_splatting_dgs_amd import network
    spec = LISTS[name]
    p = grads_of([(s, F) for s, _ in spec], seed=1, scale=1.0)
    copies = [torch.empty(s, dtype=d, device="cuda") if d != F else None for s, d in spec]
    lrs = [1e-3 * (1 + k % 5) for k in range(len(spec))]
    opt = network.Adam(p, lr=lrs, max_norm=max_norm, copies=copies)
    b1, b2 = float(np.float32(0.9)), float(np.float32(0.999))
    for t in (1, 2, 3):
        grads = grads_of(spec, seed=10 + t)
        before = [[a.cpu().double() for a in L] for L in (p, opt.exp_avg, opt.exp_avg_sq)]
        print(name, max_norm, t, flush=True)
        n = opt.step(grads)
        want = norm64(grads)
        coef = 1.0 if max_norm is None else min(1.0, max_norm / (want + 1e-6))
        assert n is None if max_norm is None else abs(float(n) - want) <= 2 * U32 * want
        for i, g in enumerate(grads):
            gd = g.cpu().double()
            ps, ms, vs, st = adam64(gd, *(L[i] for L in before), float(np.float32(lrs[i])), t, coef, b1, b2)
            m_tol = 8 * U32 * (b1 * before[1][i].abs() + (1 - b1) * coef * gd.abs()) + 2.0 ** -149
            v_tol = 10 * U32 * vs + 2.0 ** -149
            assert ((opt.exp_avg[i].cpu().double() - ms).abs() <= m_tol).all()
            assert ((opt.exp_avg_sq[i].cpu().double() - vs).abs() <= v_tol).all()
            # the step's own error: m's, half v's (8 u), and its roundings; 1 - 0.9f and 1 - 0.999f are 2^-21 off
            p_tol = U32 * ps.abs() + st.abs() * 2.0 ** -19 + \
                lrs[i] * m_tol / (1 - b1 ** t) / (torch.sqrt(vs / (1 - b2 ** t)) + 1e-8)
            assert ((p[i].cpu().double() - ps).abs() <= p_tol).all(), (i, t)
            if copies[i] is not None:
                assert torch.equal(copies[i], p[i].to(copies[i].dtype))


def test_adam_is_gs_adam_step():
    """Without clipping the step is gs_adam_step, bit for bit, rows renormalised included."""
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    shapes = [(1000, 3), (1000, 4), (1000,), (1000, 16, 3)]
    p = grads_of([(s, F) for s in shapes], seed=2, scale=1.0)
    q = [t.clone() for t in p]
    m, v = [torch.zeros_like(t) for t in q], [torch.zeros_like(t) for t in q]
    opt = network.Adam(p, lr=[1e-3, 2e-3, 3e-3, 4e-3], normalize_rows=(1,))
    for t in range(1, 4):
        g = grads_of([(s, F) for s in shapes], seed=20 + t)
        opt.step(g)
        gs.gs_adam_step([dict(param=q[i], grad=g[i], exp_avg=m[i], exp_avg_sq=v[i], rows=1000,
                              row_len=q[i].numel() // 1000, lr=1e-3 * (i + 1), normalize_rows=i == 1)
                         for i in range(4)], 0.9, 0.999, 1e-8, t)
        for a, b in zip(p + opt.exp_avg + opt.exp_avg_sq, q + m + v):
            assert torch.equal(a, b)


def test_adam_columns():
    """Column groups of one array with their own rates (SH bands), through the C entry point."""
    from differentiable_gaussian_splatting_dgs_amd import gs
    n, L = 777, 48
    p, g = grads_of([((n, L), F)], 1, 1.0)[0], grads_of([((n, L), B)], 2)[0]
    m, v, copy = torch.zeros_like(p), torch.zeros_like(p), torch.zeros(n, L, dtype=H, device="cuda")
    p0 = p.cpu().double()
    arr = (gs.GsAdamTensor * 2)()
    for a, (c0, c1, lr) in zip(arr, ((0, 3, 1e-2), (3, 45, 1e-3))):
        a.param, a.grad, a.exp_avg, a.exp_avg_sq, a.copy = (t.data_ptr() for t in (p, g, m, v, copy))
        a.rows, a.row_len, a.col_begin, a.col_end, a.lr = n, L, c0, c1, lr
        a.grad_dtype, a.copy_dtype = gs.DTYPES[B], gs.DTYPES[H]
    gs.gs_adam_step_clipped(arr, 0.9, 0.999, 1e-8, 1)
    d = (p0 - p.cpu().double())
    s = torch.sign(g.cpu().double())
    assert ((d[:, :3] - 1e-2 * s[:, :3]).abs() <= 1e-5).all() and ((d[:, 3:45] - 1e-3 * s[:, 3:45]).abs() <= 1e-5).all()
    assert (d[:, 45:] == 0).all() and (copy[:, 45:] == 0).all() and (m[:, 45:] == 0).all()
    assert torch.equal(copy[:, :45], p[:, :45].half())


def test_stream_and_graph():
    """Clip and step captured in a graph, replayed several times with eager work between, against the eager calls."""
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    spec = LISTS["mixed network"]
    grads = grads_of(spec)
    out = [torch.empty_like(g) for g in grads]
    c = network.GradClip(0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.clip(grads, out=out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.clip(grads, out=out)
    for k in range(4):
        for g, n in zip(grads, grads_of(spec, seed=30 + k, scale=0.01 + k)):
            g.copy_(n)
        print("replay", k, flush=True)
        graph.replay()
        torch.cuda.synchronize()
        e = network.GradClip(0.5)
        want = [torch.empty_like(g) for g in grads]
        e.clip(grads, out=want)
        assert torch.equal(c.state[:2], e.state[:2]) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_same_result_every_run():
    from differentiable_gaussian_splatting_dgs_amd import network
    g = grads_of(LISTS["whole chunks"])
    c = network.GradClip(0.5)
    first = float(c.norm(g))
    assert all(float(c.norm(g)) == first for _ in range(10))


def test_refusals():
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    g = grads_of([((4, 3), F), ((5,), H)])
    for bad in (-1.0, float("nan")):
        with pytest.raises(gs.GsError):
            network.GradClip(bad)
    c = network.GradClip(1.0)
    with pytest.raises(gs.GsError):
        c.norm([])
    with pytest.raises(gs.GsError):
        c.norm([g[0].cpu()])
    with pytest.raises(gs.GsError):
        c.norm([g[0].t()])
    with pytest.raises(gs.GsError):
        c.norm([g[0].double()])
    with pytest.raises(gs.GsError):
        c.clip(g, out=[g[0]])
    with pytest.raises(gs.GsError):
        c.clip(g, out=[g[0], g[1].float()])
    c.norm(g)
    with pytest.raises(gs.GsError, match="workspace"):
        gs.gs_grad_norm(g, 1.0, c.state, c.workspace[:256])
    with pytest.raises(gs.GsError):
        gs.gs_grad_norm(g, -1.0, c.state, c.workspace)
    with pytest.raises(gs.GsError):
        network.Adam([g[1]], lr=1e-3)
    with pytest.raises(gs.GsError):
        network.Adam([g[0]], lr=[1e-3, 1e-3])
    opt = network.Adam([g[0].clone()], lr=1e-3)
    with pytest.raises(gs.GsError):
        opt.step([g[1]])
    with pytest.raises(gs.GsError):
        opt.step([])

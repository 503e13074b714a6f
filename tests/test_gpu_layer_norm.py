"""Layer norm on the GPU (gs_layer_norm_fwd, gs_layer_norm_bwd, network.layer_norm) against its definition in 64 bits.

Bounds, with U = 2^-24 and u the type's unit roundoff.  The mean of n float32 numbers is within (n + 2) U mean |x| =: em
of exact (n / 4 or so in fact: the sum is a tree).  d = x - mean is off by em + U |d|.  The sum of squares is then off
by a relative (n + 6) U and, the errors of d being a common shift em, by n em^2: var by (n + 6) U var + em^2; so r is
off by a relative er = ((n + 6) U var + em^2) / (2 (var + eps)) + 4 U.  y is off by |w| r (em + |d| (er + 3 U)) and the
last sum's U, and is rounded once.  The backward's sums of g and g xh are off by (n + 4) U of their terms and by what xh
is; dx follows by the product rule."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def put(a, dtype, pad=0, lead=0):
    rows, n = a.shape
    buf = torch.full((lead + rows * (n + pad) + 16,), float("nan"), dtype=dtype, device="cuda")
    view = buf[lead:lead + rows * (n + pad)].view(rows, n + pad)[:, pad:]
    view.copy_(torch.from_numpy(a.astype(np.float32)).to(dtype))
    return view


def inputs(rows, n, dtype, seed=0, pad=0, lead=0, mean=0.5):
    rng = np.random.default_rng(seed + rows + 31 * n)
    x = put(rng.standard_normal((rows, n)) + mean, dtype, pad, lead)
    dy = put(rng.standard_normal((rows, n)) * 0.3, dtype, pad, lead)
    w = put(1 + 0.3 * rng.standard_normal((1, n)), dtype, 0, lead)[0]
    b = put(0.3 * rng.standard_normal((1, n)), dtype, 0, lead)[0]
    return x, w, b, dy


def exact(x, w, b, dy, eps):
    """y, dx, dw, db and their bounds in float64."""
    u, tiny = HALF[x.dtype], TINY[x.dtype]
    x, dy = x.double(), dy.double()
    rows, n = x.shape
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    em = (n + 2) * U * x.abs().mean(1, keepdim=True)
    er = ((n + 6) * U * var + em ** 2) / (2 * (var + eps)) + 4 * U
    xh, exh = d * r, r * (em + d.abs() * (er + 3 * U))
    y = xh * w + b
    y_err = w.abs() * exh + 2 * U * (y.abs() + (xh * w).abs()) + u * y.abs() + tiny
    g = dy * w
    flat, along = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    e_flat = (n + 4) * U * g.abs().mean(1, keepdim=True)
    e_along = (g.abs() * exh).mean(1, keepdim=True) + (n + 6) * U * (g * xh).abs().mean(1, keepdim=True) + \
        4 * er * along.abs()
    inner = g - flat - xh * along
    dx = r * inner
    dx_err = r * (e_flat + exh * along.abs() + (xh.abs() + exh) * e_along +
                  4 * U * (g.abs() + flat.abs() + (xh * along).abs())) + (er + 2 * U) * dx.abs() + u * dx.abs() + tiny
    dw, db = (dy * xh).sum(0), dy.sum(0)
    dw_err = (dy.abs() * exh).sum(0) + (rows + 4) * U * (dy * xh).abs().sum(0) + u * dw.abs() + tiny
    db_err = (rows + 4) * U * dy.abs().sum(0) + u * db.abs() + tiny
    return (y, y_err), (dx, dx_err), (dw, dw_err), (db, db_err)


def check(got, want, what):
    value, tol = want
    got = got.detach().double()
    assert got.shape == value.shape, what
    bad = ~((got - value).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - value).abs() / tol).max()))


def compare(x, w, b, dy, eps=1e-5):
    from differentiable_gaussian_splatting_dgs_amd import network
    print("norm", tuple(x.shape), x.dtype, x.stride(), w is not None, b is not None, flush=True)
    want = exact(x, w, b, dy, eps)
    check(network.layer_norm(x, w, b, eps), want[0], ("y", x.shape, x.dtype))
    torch.cuda.synchronize()
    print("backward", flush=True)
    got = network.layer_norm_backward(dy, x, w, b, eps)
    for name, g, v in zip(("dx", "dw", "db"), got, want[1:]):
        if g is not None:
            check(g, v, (name, x.shape, x.dtype))
    return got


# every kernel's widths and their edges: a thread, 1 to 64 lanes, several chunks, a block, rows read again
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 333, 500, 512, 513, 1000,
          1024, 1025, 2047, 2048, 2049, 4095, 4096, 4097, 8192, 8193, 16384, 16385, 20001]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", WIDTHS)
def test_widths(n, dtype):
    for rows in (1, 5, 67):
        x, w, b, dy = inputs(rows, n, dtype)
        compare(x, w, b, dy)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", [(100_003, 24), (30_001, 130), (4099, 768), (2000, 5000), (70_000, 3)])
def test_rows(rows, n, dtype):
    compare(*inputs(rows, n, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (8, 3), (13, 7)])
def test_strides_and_missing_weights(pad, lead, dtype):
    for rows, n in ((33, 40), (7, 129), (9, 6), (3, 4200), (2, 17000)):
        x, w, b, dy = inputs(rows, n, dtype, pad=pad, lead=lead)
        compare(x, w, b, dy)
        compare(x, None, None, dy)
        compare(x, w, None, dy)
        compare(x, None, b, dy)


@pytest.mark.parametrize("dtype", TYPES)
def test_far_means(dtype):
    """Rows whose mean is many times their spread: the squares are taken about it."""
    for n in (100, 700, 9000):
        compare(*inputs(20, n, dtype, mean=30.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_constant_rows(dtype):
    """No spread at all: eps alone is left; eps 0 makes 0 / 0."""
    from differentiable_gaussian_splatting_dgs_amd import network
    for n in (3, 32, 300, 5000, 20000):
        x = torch.full((4, n), 0.25, dtype=dtype, device="cuda")
        assert not network.layer_norm(x).any()
        assert network.layer_norm(x, eps=0.0).isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_one_bad_row(dtype):
    """A NaN or an infinity stays in its row (and in dw), whatever kernel takes it."""
    from differentiable_gaussian_splatting_dgs_amd import network
    for n in (3, 24, 200, 2000, 6000, 20000):
        for bad in (float("nan"), float("inf")):
            x, w, b, dy = inputs(9, n, dtype)
            clean = network.layer_norm(x, w, b), network.layer_norm_backward(dy, x, w, b)[0]
            x[4, n // 2] = bad
            for a, c in zip((network.layer_norm(x, w, b), network.layer_norm_backward(dy, x, w, b)[0]), clean):
                assert a[4].isnan().all() and torch.equal(a[:4], c[:4]) and torch.equal(a[5:], c[5:]), n


def test_no_rows():
    from differentiable_gaussian_splatting_dgs_amd import network
    for dtype in TYPES:
        for n in (3, 40, 9000):
            x, w, b, dy = inputs(4, n, dtype)
            assert network.layer_norm(x[:0], w, b).shape == (0, n)
            dx, dw, db = network.layer_norm_backward(dy[:0], x[:0], w, b)
            assert dx.shape == (0, n) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(dtype):
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    for rows, n in ((1000, 96), (50, 1), (70, 5), (30, 3001), (5, 30000)):
        x, w, b, dy = inputs(rows, n, dtype)
        y, (dx, dw, db) = network.layer_norm(x, w, b), network.layer_norm_backward(dy, x, w, b)
        work = torch.empty(gs.gs_layer_norm_bwd_workspace_size(x), dtype=torch.uint8, device="cuda")
        dw2, db2 = torch.empty_like(w), torch.empty_like(w)
        gs.gs_layer_norm_bwd(x, w, dy, dy, dw2, db2, work)
        assert torch.equal(dy, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)
        gs.gs_layer_norm_fwd(x, w, b, x)
        assert torch.equal(x, y)


def test_single_gradients():
    from differentiable_gaussian_splatting_dgs_amd import network
    for n in (5, 100, 5000, 20000):
        x, w, b, dy = inputs(300, n, torch.float16)
        want = network.layer_norm_backward(dy, x, w, b)
        for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
            for g, v, k in zip(network.layer_norm_backward(dy, x, w, b, need=need), want, need):
                assert (g is None) if not k else torch.equal(g, v)


def test_repeats():
    from differentiable_gaussian_splatting_dgs_amd import network
    x, w, b, dy = inputs(50_000, 100, torch.bfloat16)
    first = network.layer_norm_backward(dy, x, w, b)
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(first, network.layer_norm_backward(dy, x, w, b)))


def test_autograd_and_differences():
    from differentiable_gaussian_splatting_dgs_amd import network
    x, w, b, dy = inputs(20, 70, torch.float32)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    network.layer_norm(*leaves).backward(dy)
    want = network.layer_norm_backward(dy, x, w, b)
    assert all(torch.equal(a.grad, c) for a, c in zip(leaves, want))
    rng = np.random.default_rng(0)
    for i, leaf in enumerate(leaves):
        step = torch.from_numpy(rng.standard_normal(leaf.shape).astype(np.float32)).cuda()
        h, values = 2.0 ** -7, []
        for sign in (1, -1):
            moved = [t.detach() for t in leaves]
            moved[i] = moved[i] + sign * h * step
            values.append(float((network.layer_norm(*moved).double() * dy.double()).sum()))
        terms = leaf.grad.double() * step.double()
        # h^2 / 6 of a third derivative of the terms' size
        assert abs((values[0] - values[1]) / (2 * h) - float(terms.sum())) <= 1e-3 * float(terms.abs().sum()) + 1e-3, i
    x2 = x.clone().requires_grad_()
    network.layer_norm(x2, w, b).sum().backward()  # an expanded gradient, weights that need none
    assert torch.equal(x2.grad, network.layer_norm_backward(torch.ones_like(x), x, w, b)[0])


def test_graph_and_streams():
    from differentiable_gaussian_splatting_dgs_amd import network
    x, w, b, dy = inputs(3000, 200, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = network.layer_norm(x, w, b)
        network.layer_norm_backward(dy, x, w, b)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, network.layer_norm(x, w, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = network.layer_norm(x, w, b)
        grads = network.layer_norm_backward(dy, x, w, b)
    for i in range(3):
        for a, c in zip((x, w, b, dy), inputs(3000, 200, torch.bfloat16, seed=i + 1)):
            a.copy_(c)
        want = network.layer_norm(x, w, b), *network.layer_norm_backward(dy, x, w, b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, (y, *grads)))


def test_offsets_past_32_bits():
    from differentiable_gaussian_splatting_dgs_amd import network
    stride = 1 << 22
    buf = torch.empty(1100 * stride, dtype=torch.float16, device="cuda")
    x0, w, b, dy = inputs(1100, 100, torch.float16)
    x = torch.as_strided(buf, (1100, 100), (stride, 1))
    x.copy_(x0)
    assert torch.equal(network.layer_norm(x, w, b), network.layer_norm(x0, w, b))
    for a, c in zip(network.layer_norm_backward(x, x, w, b), network.layer_norm_backward(x0, x0, w, b)):
        assert torch.equal(a, c)

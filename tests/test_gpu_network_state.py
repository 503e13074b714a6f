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


def test_a_graph_keeps_its_clipping_buffers():
    """A clip recorded over a short list, then a longer list and tensors that take any memory that it freed: replays
    give the eager result and write nothing else."""
    from differentiable_gaussian_splatting_dgs_amd import network
    new = make(1)
    grads = [new(50, 3), new(77)]
    out = [torch.empty_like(g) for g in grads]
    c = network.GradClip(0.5)
    c.clip(grads, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.clip(grads, out=out)
    state = c.state
    many = [new(3) for _ in range(200)]
    c.clip(many, out=[torch.empty_like(g) for g in many])
    filled = [torch.full((n,), 7.0, device="cuda") for n in (4, 64, 2048, 2112, 4096, 8192) for _ in range(64)]
    for k in range(4):
        for g in grads:
            g.copy_(new(*g.shape) * (k + 0.01))
        print("replay", k, flush=True)
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(g) for g in grads]
        e = network.GradClip(0.5)
        e.clip(grads, out=want)
        assert torch.equal(state[:2], e.state[:2]) and all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(bool((t == 7).all()) for t in filled)


def test_clips_on_two_streams():
    """One GradClip on two streams with no order between them: each call's coefficient is its own list's."""
    from differentiable_gaussian_splatting_dgs_amd import network
    new = make(2)
    lists = [[new(1 << 20) * 1e-4, new(5000)], [new(300_000) * 30, new(64), new(7)]]
    outs = [[torch.empty_like(g) for g in grads] for grads in lists]
    want = [[torch.empty_like(g) for g in grads] for grads in lists]
    for grads, w in zip(lists, want):
        network.GradClip(0.1).clip(grads, out=w)
    c = network.GradClip(0.1)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, grads, out in zip(streams, lists, outs):
            with torch.cuda.stream(s):
                c.clip(grads, out=out)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.fixture
def elsewhere(monkeypatch):
    """Another device than the tensors' is the current one, as far as the calls can tell; the devices they enter."""
    from differentiable_gaussian_splatting_dgs_amd import gs
    now, entered = [1], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)
            now.append(self.index)

        def __exit__(self, *a):
            now.pop()

    monkeypatch.setattr(gs, "_current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    return entered


def test_calls_go_to_their_tensors_device(elsewhere):
    """Each call enters its tensors' device before it takes a stream, once."""
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    new = make(3)
    x, w, b, dy = new(40, 24), new(20, 24), new(20), new(40, 20)
    grads = [new(30, 3), new(9)]
    c = network.GradClip(0.5)
    opt = network.Adam([new(30, 3), new(9)], lr=1e-2, max_norm=0.5)
    for name, call in (("linear", lambda: network.linear(x, w, b, act="silu")),
                       ("backward", lambda: network.linear_backward(dy, x, w, b, act="silu")),
                       ("norm", lambda: c.norm(grads)),
                       ("clip", lambda: c.clip(grads, out=[torch.empty_like(g) for g in grads])),
                       ("adam", lambda: opt.step(grads)),
                       ("gs norm", lambda: gs.gs_grad_norm(grads, 0.5, c.state, c.workspace)),
                       ("gs clip", lambda: gs.gs_grad_clip(grads, grads, 0.5, c.state, c.workspace))):
        del elsewhere[:]
        print(name, flush=True)
        call()
        assert elsewhere == [0], name


def test_tensors_of_several_devices_are_refused():
    from differentiable_gaussian_splatting_dgs_amd import gs, network
    new = make(4)
    p = [new(5), new(3)]
    with pytest.raises(gs.GsError):
        network.Adam(p, lr=1e-3, exp_avg=[torch.zeros(5), torch.zeros(3)])
    opt = network.Adam(p, lr=1e-3)
    with pytest.raises(gs.GsError):
        opt.step([g.cpu() for g in p])
    c = network.GradClip(1.0)
    for bad in ([None], [p[0].cpu()], [p[0], p[1].cpu()], []):
        for call in (c.norm, c.clip):
            with pytest.raises(gs.GsError):
                call(bad)
    c.norm(p)
    with pytest.raises(gs.GsError):
        gs.gs_grad_norm(p, 1.0, c.state.cpu(), c.workspace)
    with pytest.raises(gs.GsError):
        gs.gs_grad_clip(p, p, 1.0, c.state, c.workspace.cpu())


def test_a_backward_after_the_step_is_refused():
    """The gradients of a layer whose weights a step has changed since would be those of other weights."""
    from differentiable_gaussian_splatting_dgs_amd import network
    new = make(5)
    x, w = new(20, 8), new(6, 8)
    c = w.to(H).requires_grad_()
    opt = network.Adam([w], lr=1e-2, max_norm=1.0, copies=[c])
    y = network.linear(x.to(H).requires_grad_(), c, act="silu").float().sum()
    opt.step([new(6, 8).to(H)])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    y = network.linear(x.to(H).requires_grad_(), c, act="silu").float().sum()
    y.backward()
    opt.step([c.grad])

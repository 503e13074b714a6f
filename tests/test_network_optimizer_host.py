"""What network.Adam hands to the library, looked at on the CPU: the calls are replaced by recorders."""
import gc
import struct
import weakref

import pytest
import torch

from differentiable_gaussian_splatting_dgs_amd import gs, network

FIELDS = ("param", "grad", "exp_avg", "exp_avg_sq", "copy", "rows", "row_len", "copy_dtype", "normalize_rows")


@pytest.fixture
def calls(monkeypatch):
    """The descriptors of every gs_adam_step_clipped call."""
    seen = []

    def pointer(t, dtype=None, name="tensor"):
        if t is None:
            return None
        if not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
            raise gs.GsError(name)
        return t.data_ptr()

    def table(grads, out):
        return struct.pack("=%dq" % (4 * len(grads)),
                           *[v for g in grads for v in (g.data_ptr(), 0, g.numel(), gs.DTYPES[g.dtype])])

    monkeypatch.setattr(gs, "_p", pointer)
    monkeypatch.setattr(gs, "_grad_table", table)
    monkeypatch.setattr(gs, "gs_adam_step_clipped",
                        lambda t, *a, **k: seen.append([{f: getattr(e, f) for f in FIELDS} for e in t]))
    return seen


def optimizer():
    p = [torch.randn(6, 4), torch.randn(5)]
    return network.Adam(p, lr=[1e-3, 2e-3], copies=[p[0].half(), None], normalize_rows=(0,))


def expect(opt, grads, got):
    for i, e in enumerate(got):
        want = dict(param=opt.params[i], grad=grads[i], exp_avg=opt.exp_avg[i], exp_avg_sq=opt.exp_avg_sq[i],
                    copy=opt.copies[i])
        assert {k: e[k] or None for k in want} == {k: None if t is None else t.data_ptr() for k, t in want.items()}
        assert e["rows"] * e["row_len"] == opt.params[i].numel()
        assert e["row_len"] == (opt.params[i].shape[-1] if i in (0,) else 1)
        if opt.copies[i] is not None:
            assert e["copy_dtype"] == gs.DTYPES[opt.copies[i].dtype]


def replace(opt, what):
    if what == "data":  # what module.to() and loaders do to a parameter
        opt.params[0].data = torch.randn(6, 4)
    elif what == "longer":
        opt.params[1] = torch.randn(9)
        opt.exp_avg[1], opt.exp_avg_sq[1] = torch.zeros(9), torch.zeros(9)
    elif what == "moment":
        opt.exp_avg[0] = torch.ones(6, 4)
    elif what == "second moment":
        opt.exp_avg_sq[1].data = torch.ones(5)
    elif what == "copy":
        opt.copies[0] = opt.copies[0].bfloat16()
    elif what == "copy's data":
        opt.copies[0].data = torch.zeros(6, 4, dtype=torch.float16)
    elif what == "no copy":
        opt.copies[0] = None
    elif what == "new copy":
        opt.copies[1] = torch.zeros(5, dtype=torch.float16)
    elif what == "shape":  # other rows in the same memory
        for t in (opt.params[0], opt.exp_avg[0], opt.exp_avg_sq[0], opt.copies[0]):
            t.data = t.data.view(3, 8)


@pytest.mark.parametrize("what", ["nothing", "data", "longer", "moment", "second moment", "copy", "copy's data", "no copy",
                                  "new copy", "shape"])
def test_a_step_takes_what_the_lists_hold(calls, what):
    opt = optimizer()
    for k in range(3):
        if k == 1:
            replace(opt, what)
        grads = [torch.randn(p.shape) for p in opt.params]
        opt.step(grads)
        expect(opt, grads, calls[-1])
    assert opt.t == len(calls) == 3
    assert [e.lr for e in opt.table] == [pytest.approx(1e-3), pytest.approx(2e-3)]


def test_the_table_holds_its_memory(calls):
    """The storages that the table names live until it names others: nothing else can be allocated there."""
    opt = optimizer()
    opt.params[0].data = torch.randn(6, 4)
    freed = opt._held[0].data_ptr()
    assert opt.table[0].param == freed != opt.params[0].data_ptr()
    opt.step([torch.randn(p.shape) for p in opt.params])
    assert opt._held[0].data_ptr() == opt.table[0].param == opt.params[0].data_ptr()


@pytest.mark.parametrize("list_name,bad", [("params", torch.zeros(6, 4, dtype=torch.float64)), ("params", torch.zeros(4, 6).t()),
                                           ("params", None), ("exp_avg", None), ("copies", "half"),
                                           ("exp_avg", torch.zeros(6, 3)), ("exp_avg_sq", torch.zeros(4, 6).t()),
                                           ("copies", torch.zeros(24, dtype=torch.float16)),
                                           ("copies", torch.zeros(6, 4, dtype=torch.int32))])
def test_replacements_are_checked(calls, list_name, bad):
    opt = optimizer()
    grads = [torch.randn(p.shape) for p in opt.params]
    opt.step(grads)
    kept = getattr(opt, list_name)[0]
    getattr(opt, list_name)[0] = bad
    with pytest.raises(gs.GsError):
        opt.step(grads)
    assert len(calls) == 1 and opt.t == 1
    getattr(opt, list_name)[0] = kept
    opt.step(grads)
    expect(opt, grads, calls[-1])


def test_a_transposed_view_is_refused(calls):
    """Same address, same shape, another order."""
    opt = network.Adam([torch.randn(4, 4)], lr=1e-3)
    opt.step([torch.randn(4, 4)])
    opt.params[0].data = opt.params[0].data.t()
    with pytest.raises(gs.GsError):
        opt.step([torch.randn(4, 4)])


def test_lists_of_another_length(calls):
    opt = optimizer()
    opt.exp_avg.append(torch.zeros(5))
    with pytest.raises(gs.GsError):
        opt.step([torch.randn(p.shape) for p in opt.params])
    with pytest.raises(gs.GsError):
        network.Adam([torch.tensor(1.0)], lr=1e-3, normalize_rows=(0,))


@pytest.fixture
def clip_calls(monkeypatch):
    """Every gs_grad_norm call's state and workspace, with the stream and the capture that `at` says."""
    seen, at = [], dict(stream=1, capturing=False)
    monkeypatch.setattr(gs, "_grad_table", lambda grads, out: b"")
    monkeypatch.setattr(gs, "grad_norm_table", lambda n, t, m, state, ws: seen.append((state, ws)))
    monkeypatch.setattr(gs, "_raw_stream", lambda device: at["stream"])
    monkeypatch.setattr(gs, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at["capturing"])
    return seen, at


def shared(a, b):
    return any(x.data_ptr() == y.data_ptr() for x, y in zip(a, b))


def test_recorded_calls_keep_their_buffers(clip_calls):
    """A longer list, or another recording, neither frees nor uses what a recorded call uses."""
    seen, at = clip_calls
    c = network.GradClip(1.0)
    one, many = [torch.ones(2)], [torch.ones(2)] * 200
    c.norm(one)
    for _ in range(2):
        at["capturing"] = True
        c.norm(one)
        at["capturing"] = False
        c.norm(many)
        c.norm(one)
    eager, recorded = [seen[k] for k in (0, 2, 3, 5, 6)], [seen[k] for k in (1, 4)]
    pointers = [[t.data_ptr() for t in r] for r in recorded]
    refs = [[weakref.ref(t) for t in r] for r in recorded]
    assert not shared(*recorded) and not any(shared(r, e) for r in recorded for e in eager)
    del seen[:], eager, recorded
    gc.collect()
    assert [[r().data_ptr() for r in p] for p in refs] == pointers


def test_streams_have_their_own_buffers(clip_calls):
    seen, at = clip_calls
    c = network.GradClip(1.0)
    for stream in (1, 2, 1, 2):
        at["stream"] = stream
        c.norm([torch.ones(2)])
        assert c.state is seen[-1][0] and c.workspace is seen[-1][1]
    assert not shared(seen[0], seen[1])
    for k in (0, 1):
        assert all(x is y for x, y in zip(seen[k], seen[k + 2]))


def test_a_longer_list_gets_a_longer_workspace(clip_calls):
    seen, _ = clip_calls
    c = network.GradClip(1.0)
    for n in (1, 200, 3, 65):
        c.norm([torch.ones(2)] * n)
        assert seen[-1][1].numel() >= gs.gs_grad_workspace_size(n)
    assert seen[1][1] is seen[2][1] is seen[3][1] and all(s[0] is seen[0][0] for s in seen)


def test_a_step_counts_as_a_change(calls):
    """Autograd knows that a step wrote parameters and copies: a graph that saved them refuses a backward."""
    opt = optimizer()
    w, c = opt.params[1].requires_grad_(), opt.copies[0].requires_grad_()
    loss = w.square().sum() + c.square().sum().float()
    opt.step([torch.randn(p.shape) for p in opt.params])
    assert w._version == 1 and c._version == 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("inference", [False, True])
def test_a_clip_counts_as_a_change(clip_calls, monkeypatch, inference):
    monkeypatch.setattr(gs, "gs_grad_clip", lambda *a: None)
    with torch.inference_mode(inference):
        g, out = [torch.ones(2), torch.ones(3)], [torch.ones(2), torch.ones(3)]
        c = network.GradClip(1.0)
        c.norm(g)
        if not inference:  # tensors made in inference mode have no versions
            assert [t._version for t in g] == [0, 0]
        c.clip(g, out=out)
        c.clip(g)
        if not inference:
            assert [t._version for t in g + out] == [1, 1, 1, 1]


def test_a_copy_of_another_type_in_the_same_memory(calls):
    opt = optimizer()
    grads = [torch.randn(p.shape) for p in opt.params]
    opt.step(grads)
    opt.copies[0] = opt.copies[0].view(torch.bfloat16)
    opt.step(grads)
    assert calls[0][0]["copy"] == calls[1][0]["copy"]
    expect(opt, grads, calls[1])


@pytest.mark.parametrize("name", ["exp_avg", "exp_avg_sq", "copies"])
def test_transposed_moments_and_copies_are_refused(calls, name):
    """The parameter's address, shape and type, another order."""
    p = torch.randn(4, 4)
    opt = network.Adam([p], lr=1e-3, copies=[p.half()])
    opt.step([torch.randn(4, 4)])
    getattr(opt, name)[0].data = getattr(opt, name)[0].data.t()
    with pytest.raises(gs.GsError):
        opt.step([torch.randn(4, 4)])

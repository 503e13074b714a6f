"""Networks beside the Gaussians: the fused linear layer with its gradients, gradient
clipping by the global norm, and an Adam optimizer that takes the clipping
coefficient on the device.

A network's rows are Gaussians (features decoded to Gaussian parameters, offsets for
a time step) or views (an appearance code per camera); its outputs go to
`gs.rasterize` and its gradients come back through it.  Plumbing over the C ABI
(gs_linear_*, gs_grad_*, gs_adam_step_clipped): buffers and the order of the calls.
"""
from __future__ import annotations

import contextlib
import ctypes as C

import numpy as np
import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import gs
from .gs import GsError


def _workspace(nbytes, device):
    """uint8 tensor of nbytes, 256-byte aligned."""
    t = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-t.data_ptr()) % 256
    return t[off:off + nbytes]


def linear_backward(dy, x, w, bias=None, act="none", need=(True, True, True)):
    """dx, dw, db of y = act(x w^T + bias) from dy = dL/dy (None where need is False; db None without a bias).
    The gradient of a residual added to y is dy itself."""
    need_dx, need_dw, need_db = need
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_dx else None
    dw = torch.empty_like(w, memory_format=torch.contiguous_format) if need_dw else None
    db = torch.empty_like(bias, memory_format=torch.contiguous_format) if need_db and bias is not None else None
    gs.linear_bwd_into(x, w, bias, dy, dx, dw, db, None, act)
    return dx, dw, db


class LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, act):
        ctx.act, ctx.has_bias = act, bias is not None
        ctx.save_for_backward(x, w, bias)
        return gs.linear_fwd_into(x, w, bias, residual, None, act)

    @staticmethod
    def backward(ctx, dy):
        x, w, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            grads = linear_backward(_plain_rows(dy), x, w, bias, ctx.act, need[:3])
            dx, dw, db = gs.differentiated_once("network.linear", grads, (dy, x, w, bias))
        return dx, dw, db, dy if need[3] else None, None


def _plain_rows(t):
    """t if its rows are contiguous and do not overlap, else a contiguous copy."""
    s0, s1 = t.stride()
    return t if (s1 == 1 or t.shape[1] <= 1) and (s0 >= t.shape[1] or t.shape[0] <= 1) else t.contiguous()


def linear(x, w, bias=None, residual=None, act="none"):
    """act(x w^T + bias) + residual, differentiable in all four tensors, once: a second derivative (a penalty on a
    gradient) raises GsError, but for the residual's.  Forward mode raises NotImplementedError.

    x [rows, n_in], w [n_out, n_in], bias [n_out], residual [rows, n_out], all of one type (float32, float16 or
    bfloat16); x and residual may have strided rows, which must not overlap (but the residual may be one row expanded).
    act: "none", "relu", "silu" or "gelu" (tanh form)."""
    # under forward mode a tensor with a tangent need not require a gradient: the function raises for it
    if forward_ad._current_level >= 0 or torch.is_grad_enabled() and (
            x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad) or
            (residual is not None and residual.requires_grad)):
        return LinearFunction.apply(x, w, bias, residual, act)
    return gs.linear_fwd_into(x, w, bias, residual, None, act)


_HERE = contextlib.nullcontext()


def _device_of(grads):
    """A context in which the gradients' device is the current one."""
    if not grads:
        raise GsError("no gradients")
    if not isinstance(grads[0], torch.Tensor):
        raise GsError("gradients must be tensors")
    return _on(grads[0].get_device())


def _on(device):
    """A context in which that device is the current one (-1, the host: nothing; the calls refuse its tensors)."""
    return _HERE if device < 0 or device == gs._current_device() else torch.cuda.device(device)


class GradClip:
    """Clipping of gradient lists to a global norm; owns the clipping state and the workspace.

    norm() and clip() return the norm before clipping as a float32 device scalar (overwritten by the stream's next
    call); nothing synchronises.  Every stream has a state and a workspace of its own, so calls on several streams need
    no order between them, and so has every call that is recorded into a graph: its replays use them for as long as
    the GradClip lives, which has to be as long as the graph does.  `state` is the last call's."""

    def __init__(self, max_norm):
        self.max_norm = float(max_norm)
        if not self.max_norm >= 0:
            raise GsError("max_norm must be >= 0")
        self.state = None
        self._of_stream = {}  # (device, stream): state, value, workspace, the tensors that it is for
        self._recorded = []

    def _prepare(self, grads):
        n, device = len(grads), grads[0].device
        recorded = torch.cuda.is_current_stream_capturing()
        key = device, gs._raw_stream(gs._current_device())
        held = None if recorded else self._of_stream.get(key)
        if held is None or held[3] < n:
            workspace = _workspace(gs.gs_grad_workspace_size(n), device)
            if held is None:
                state = torch.empty(gs.CLIP_STATE_FLOATS, dtype=torch.float32, device=device)
                held = state, state[0], workspace, n
            else:  # the old workspace goes back to this stream, behind the work that uses it
                held = held[0], held[1], workspace, n
            if recorded:
                self._recorded.append(held)
            else:
                self._of_stream[key] = held
        self.state, self.value, self.workspace, _ = held

    def norm(self, grads, table=None):
        """The global norm of the list; the coefficient is left in state[1] for gs_adam_step_clipped.  table: the
        list's packed descriptors, if the caller has them."""
        with _device_of(grads):
            table = gs._grad_table(grads, None) if table is None else table
            self._prepare(grads)
            gs.grad_norm_table(len(grads), table, self.max_norm, self.state, self.workspace)
            return self.value

    def clip(self, grads, out=None):
        """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or into out."""
        with _device_of(grads):
            self._prepare(grads)
            out = grads if out is None else out
            gs.gs_grad_clip(grads, out, self.max_norm, self.state, self.workspace)
            increment_version(out)
            return self.value


class Adam:
    """Adam over float32 parameters with the gradients clipped to a global norm, in two passes: the norm, then the
    update that takes its coefficient on the device.

    params: float32 device tensors, updated in place.  lr: one rate, or one for each parameter.  copies: for each
    parameter None or a 16-bit tensor of its shape that receives the updated values (the tensor a 16-bit network
    computes with).  normalize_rows: indices of parameters whose rows are renormalised to unit length after the
    update (quaternions).  exp_avg, exp_avg_sq: the moments, zeros by default.  A step takes what the lists params,
    exp_avg, exp_avg_sq and copies hold at that time: their entries and the entries' data may be replaced (moments
    restored, `p.data = ...`).  A step whose norm is not finite changes nothing on the device; it still counts in
    `t`.  Recorded into a graph, a step keeps its number: replays correct the moments' bias by it."""

    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, max_norm=None, copies=None, normalize_rows=(),
                 exp_avg=None, exp_avg_sq=None):
        self.params = list(params)
        n = len(self.params)
        lrs = [float(lr)] * n if isinstance(lr, (int, float)) else [float(v) for v in lr]
        self.copies = [None] * n if copies is None else list(copies)
        self.exp_avg = [torch.zeros_like(p) for p in self.params] if exp_avg is None else list(exp_avg)
        self.exp_avg_sq = [torch.zeros_like(p) for p in self.params] if exp_avg_sq is None else list(exp_avg_sq)
        if not (len(lrs) == len(self.copies) == len(self.exp_avg) == len(self.exp_avg_sq) == n):
            raise GsError("lr, copies and the moments need one entry for each parameter")
        self.betas, self.eps, self.t = (float(betas[0]), float(betas[1])), float(eps), 0
        self.clipper = None if max_norm is None else GradClip(max_norm)
        self.normalize_rows = frozenset(normalize_rows)
        self.table = (gs.GsAdamTensor * max(n, 1))()
        for a, v in zip(self.table, lrs):
            a.lr = v
        # the two fields that change from step to step
        size, field = C.sizeof(gs.GsAdamTensor), gs.GsAdamTensor
        self._grad_words = np.frombuffer(self.table, dtype=np.int64)[field.grad.offset // 8::size // 8][:n]
        self._dtype_words = np.frombuffer(self.table, dtype=np.int32)[field.grad_dtype.offset // 4::size // 4][:n]
        self._describe()

    def _places(self):
        """Where every tensor lies and whether it is contiguous, the copies' types and the lengths of the rows to
        renormalise: what a step compares with the table."""
        copies = [c for c in self.copies if c is not None]
        tensors = [*self.params, *self.exp_avg, *self.exp_avg_sq, *copies]
        try:
            return ([*map(torch.Tensor.data_ptr, tensors)], all(map(torch.Tensor.is_contiguous, tensors)),
                    [c if c is None else c.dtype for c in self.copies],
                    self.normalize_rows and [p.shape for i, p in enumerate(self.params) if i in self.normalize_rows])
        except (TypeError, AttributeError):
            raise GsError("parameters, moments and copies must be tensors") from None

    def _describe(self):
        """Checks parameters, moments and copies and writes their places and sizes into the table.  The detached
        tensors hold the memory that the table names for as long as it does: a tensor at the same address in a later
        step is in that memory."""
        n = len(self.params)
        if not len(self.exp_avg) == len(self.exp_avg_sq) == len(self.copies) == n == len(self._dtype_words):
            raise GsError("copies and the moments need one entry for each parameter")
        described, rows = self._places(), []
        for i, (p, m, v, c) in enumerate(zip(self.params, self.exp_avg, self.exp_avg_sq, self.copies)):
            at = [gs._p(p, torch.float32, f"parameter {i}")]
            for t, k in ((m, "exp_avg"), (v, "exp_avg_sq")):
                at.append(gs._p(t, torch.float32, f"{k} {i}"))
                if t.shape != p.shape:
                    raise GsError(f"{k} {i} must have its parameter's shape")
            at.append(gs._p(c, None, f"copy {i}"))
            if c is not None and (c.shape != p.shape or c.dtype not in gs.DTYPES):
                raise GsError(f"copy {i} must have its parameter's shape and a floating type")
            if any(t is not None and t.get_device() != self.params[0].get_device() for t in (p, m, v, c)):
                raise GsError("parameters, moments and copies must be on one device")
            unit = i in self.normalize_rows
            if unit and p.dim() == 0:
                raise GsError(f"parameter {i} has no rows to renormalise")
            row_len = p.shape[-1] if unit else 1
            rows.append((at, gs.DTYPES[c.dtype] if c is not None else 0, unit, row_len, p.numel() // max(row_len, 1)))
        for a, (at, copy_dtype, unit, row_len, count) in zip(self.table, rows):
            a.param, a.exp_avg, a.exp_avg_sq, a.copy = at
            a.copy_dtype, a.normalize_rows, a.row_len, a.col_end, a.rows = copy_dtype, unit, row_len, row_len, count
        self._shapes = [p.shape for p in self.params]
        self._described = described
        self._held = [t.detach() for tensors in (self.params, self.exp_avg, self.exp_avg_sq, self.copies)
                      for t in tensors if t is not None]

    def step(self, grads):
        """One step with gradients grads (float32 or 16-bit, contiguous).  Returns the global norm before clipping
        as a float32 device scalar (None without max_norm)."""
        if len(grads) != len(self.params):
            raise GsError(f"{len(self.params)} parameters, {len(grads)} gradients")
        packed = gs._grad_table(grads, None)
        if self._places() != self._described:
            self._describe()
        for g, p, shape in zip(grads, self.params, self._shapes):
            if g.shape != shape:
                if g.shape != p.shape:
                    raise GsError("a gradient must have its parameter's shape")
                self._describe()  # another shape in the same memory
        if grads and grads[0].get_device() != self.params[0].get_device():
            raise GsError("gradients must be on their parameters' device")
        words = np.frombuffer(packed, dtype=np.int64).reshape(-1, 4)  # grad, out, count, dtype
        self._grad_words[:] = words[:, 0]
        self._dtype_words[:] = words[:, 3]
        if not self.params:
            self.t += 1
            return None
        with _on(self.params[0].get_device()):
            norm = self.clipper.norm(grads, packed) if self.clipper is not None else None
            self.t += 1
            gs.gs_adam_step_clipped(self.table, self.betas[0], self.betas[1], self.eps, self.t,
                                    self.clipper.state if self.clipper is not None else None)
            # a graph that saved one of them must not go backward on the new values
            increment_version(self.params + [c for c in self.copies if c is not None])
        return norm

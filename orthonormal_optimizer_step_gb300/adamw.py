"""AdamW over many tensors and the norm of their gradients (C ABI in include/dion_adamw.h).

For what the orthonormal step does not take: embeddings, output heads, norm
weights, biases.  A plan holds the list of tensors, checked once, as the table
that the library reads; a program makes it when it sets up its optimizer and
keeps it.  `set_gradients` gives it new gradient tensors where a program does
not keep theirs (a step captured before that reads the old ones' memory, which the
program has to keep then).  All tensors of a plan are on one device, which is the
current one when a call uses it.

These checks are host time: for 65 tensors a plan takes 0.6 to 1 ms, a gradient
list 0.12 and `set_gradients` 0.2, beside calls of 6 to 9 us.  A program whose
gradients are new tensors in each step pays the last one in each step; one that
zeroes them in place does not.

    first, second = dion_adamw_state(params, bits=8)             # or 32
    plan = dion_adamw_plan(params, grads, first, second)
    norm = dion_grad_norm(plan, max_norm=1.0)                    # (norm, factor) on the device
    dion_adamw_step(plan, step=t, lr=1e-3, weight_decay=0.1, grad_scale=norm[1:])

Parameters are updated in place, behind autograd's back: a plan's tensors carry
no record of it, and a graph that holds an old value is not warned.  A plan goes
with the memory that its tensors had when it was made, and keeps that memory: a
parameter that is given other memory later (p.data = ...) needs a new plan.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch
from torch import empty

import orthonormal_optimizer_step_gb300 as _od
from orthonormal_optimizer_step_gb300.q8 import _cuda, _current_device, _raw_stream, _same_device, _type

BLOCK = 256                       # values of an 8-bit state that share a scale
_E4M3, _F32, _BF16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16


class State8(NamedTuple):
    """An 8-bit state of a tensor: E4M3 values in its shape, a float32 scale for each 256 of them in memory order."""
    data: torch.Tensor
    scale: torch.Tensor


class _Tensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_longlong), ("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("p_type", ctypes.c_int), ("g_type", ctypes.c_int),
                ("lr_factor", ctypes.c_float), ("decay_factor", ctypes.c_float)]


def _flat(t, n, what):
    """The address of a tensor of n values without gaps."""
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} values, expected {n}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _of_length(items, count, what):
    items = list(items)
    if len(items) != count:
        raise ValueError(f"{len(items)} {what} for {count} tensors")
    return items


class GradList:
    """A list of gradients for dion_grad_norm (see dion_grad_list)."""

    def __init__(self, grads):
        grads = list(grads)
        self.count = len(grads)
        self.table = (_Tensor * self.count)()
        # the memory that the table points to is kept alive, and nothing else: aliases, since a tensor that a program
        # gives other memory (p.data = ...) would let go of it
        self.tensors = [[g.detach() for g in grads]]
        self.device = None
        for i, g in enumerate(grads):
            self._gradient(i, g, g.numel())
        self._workspace_bytes = self._needs()

    def _needs(self):
        """Workspace bytes of the norm: 0 where the library uses none (should its limit be lower, its answer says so)."""
        if self.count <= 256 and sum(e.n + 2047 >> 11 for e in self.table) <= 512:
            return 0
        return dion_grad_norm_workspace_size(self.count)

    def _gradient(self, i, g, n):
        e = self.table[i]
        dev = _cuda(g, f"gradient {i}")
        if self.device is None:
            self.device = dev
        elif dev != self.device:
            raise ValueError(f"gradient {i} is on cuda:{dev}, expected cuda:{self.device}")
        e.g_type = _type(g.dtype, f"gradient {i}")
        e.g = _flat(g, n, f"gradient {i}")
        e.n = n

    def _use(self):
        """The table's address for a call; its tensors have to be on the current device."""
        if self.device is not None and self.device != _current_device():
            raise ValueError(f"the tensors are on cuda:{self.device}, but the current device is cuda:{_current_device()}")
        return self.table


class AdamWPlan(GradList):
    """The tensors of dion_adamw_step (see dion_adamw_plan)."""

    def __init__(self, params, grads, first, second, copies, lr_factors, decay_factors):
        params = list(params)
        count = len(params)
        grads, first, second = (_of_length(t, count, what) for t, what in (
            (grads, "gradients"), (first, "first moments"), (second, "second moments")))
        copies = _of_length(copies, count, "copies") if copies is not None else [None] * count
        lr_factors = _of_length(lr_factors, count, "learning rate factors") if lr_factors is not None else [1.0] * count
        decay_factors = _of_length(decay_factors, count, "weight decay factors") if decay_factors is not None else [1.0] * count
        for i, (p, g) in enumerate(zip(params, grads)):
            if g.shape != p.shape:
                raise ValueError(f"gradient {i} must have its parameter's shape")
        super().__init__(grads)
        self.tensors += [[t.detach() for t in params], *([State8(*(x.detach() for x in t)) if isinstance(t, State8) else t.detach()
                                                          for t in moments] for moments in (first, second)),
                         [t if t is None else t.detach() for t in copies]]
        written = []
        for i in range(count):
            p, m, v, c, e = params[i], first[i], second[i], copies[i], self.table[i]
            n = e.n
            _same_device(self.device, **{f"parameter {i}": p})
            e.p_type = _type(p.dtype, f"parameter {i}")
            e.p = _flat(p, n, f"parameter {i}")
            written.append((e.p, n * p.element_size(), f"parameter {i}"))
            if isinstance(m, State8) is not isinstance(v, State8):
                raise TypeError(f"the moments of tensor {i} must both be float32 or both State8")
            for t, name, what in ((m, "m", "first"), (v, "v", "second")):
                what = f"{what} moment {i}"
                data, scale = t if isinstance(t, State8) else (t, None)
                dtype = _F32 if scale is None else _E4M3
                if data.dtype is not dtype:
                    raise TypeError(f"{what} must be {dtype}, got {data.dtype}")
                _same_device(self.device, **{what: data, f"{what}'s scale": scale})
                setattr(e, name, _flat(data, n, what))
                written.append((getattr(e, name), n * data.element_size(), what))
                if scale is not None:
                    if scale.dtype is not _F32:
                        raise TypeError(f"{what}: scales must be float32, got {scale.dtype}")
                    at = _flat(scale, -(-n // BLOCK), f"{what}'s scale")
                    setattr(e, name + "_scale", at)
                    written.append((at, 4 * scale.numel(), f"{what}'s scale"))
            if c is not None:
                if p.dtype is not _F32 or c.dtype is not _BF16:
                    raise TypeError(f"copy {i} must be bfloat16, of a float32 parameter")
                _same_device(self.device, **{f"copy {i}": c})
                e.copy = _flat(c, n, f"copy {i}")
                written.append((e.copy, 2 * n, f"copy {i}"))
            e.lr_factor, e.decay_factor = lr_factors[i], decay_factors[i]
            if not math.isfinite(e.lr_factor) or not math.isfinite(e.decay_factor):
                raise ValueError(f"the factors of tensor {i} must be finite")
        self._written = sorted(x for x in written if x[1])
        for (a, size, one), (b, _, other) in zip(self._written, self._written[1:]):
            if a + size > b:
                raise ValueError(f"{one} and {other} share memory")
        self._apart()
        self._workspace = None

    def _apart(self):
        """No gradient lies in what a step writes."""
        every = sorted(self._written + [(e.g, e.n * (2 if e.g_type else 4), None) for e in self.table if e.n], key=lambda x: x[:2])
        end, last = 0, None                        # of what is written so far, and of the gradients
        gend = 0
        for at, size, what in every:
            if at < end or (what is not None and at < gend):
                raise ValueError(f"a gradient shares memory with {what or last}")
            if what is None:
                gend = max(gend, at + size)
            else:
                end, last = at + size, what

    def set_gradients(self, grads):
        """Other gradient tensors, of the same shapes, for the calls that follow."""
        grads = _of_length(grads, self.count, "gradients")
        old, before = self.tensors[0], [(e.g, e.g_type) for e in self.table]
        try:
            for i, (p, g) in enumerate(zip(self.tensors[1], grads)):
                if g.shape != p.shape:
                    raise ValueError(f"gradient {i} must have its parameter's shape")
                self._gradient(i, g, p.numel())
            self._apart()
        except Exception:
            for e, (e.g, e.g_type) in zip(self.table, before):
                pass
            self.tensors[0] = old
            raise
        self.tensors[0] = [g.detach() for g in grads]


def dion_grad_list(grads):
    """A list of gradients (float32 or bfloat16) as dion_grad_norm takes it; AdamW plans are taken as well."""
    return GradList(grads)


def dion_adamw_state(params, *, bits=32):
    """Zeroed first and second moments of the parameters: float32 tensors, or State8 with bits=8."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits!r}")

    def new(p):
        if bits == 32:
            return torch.zeros_like(p, dtype=_F32, memory_format=torch.contiguous_format, requires_grad=False)
        data = torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(_E4M3)
        return State8(data, torch.zeros(-(-p.numel() // BLOCK), dtype=_F32, device=p.device))

    params = list(params)
    return [new(p) for p in params], [new(p) for p in params]


def dion_adamw_plan(params, grads, first, second, *, copies=None, lr_factors=None, decay_factors=None):
    """The tensors of dion_adamw_step, checked once.

    params, grads: contiguous float32 or bfloat16 tensors, in any mixture; first,
    second: their moments (dion_adamw_state), where second[i] holds v in float32 or
    sqrt(v) in 8 bits; copies: bfloat16 tensors that receive the new float32
    parameters, or None each; lr_factors, decay_factors: a number for each tensor
    that multiplies lr and weight_decay (0 for a norm's weight, say).  Nothing that
    a step writes may share memory with another tensor of the plan."""
    return AdamWPlan(params, grads, first, second, copies, lr_factors, decay_factors)


def dion_grad_norm_workspace_size(count: int) -> int:
    out = ctypes.c_size_t(0)
    _od._check(_od.lib().dion_grad_norm_workspace_size(count, ctypes.byref(out)), "dion_grad_norm_workspace_size")
    return out.value


def dion_grad_norm(grads, *, max_norm=math.inf, out=None, workspace=None, stream=None):
    """(norm, factor) of all gradients of a list or plan, float32 on the device.

    factor = min(1, max_norm / (norm + 1e-6)); NaN where the norm is not finite,
    with which dion_adamw_step does nothing.  Squares are float32 (gradients from 2e-23 to
    1.8e19 count), sums float64 in a fixed order."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_grad_norm(grads, max_norm=max_norm, out=out, workspace=workspace)
    table, dev = grads._use(), grads.device
    if dev is None:
        dev = _current_device()
    device = torch.device("cuda", dev)
    if out is None:
        out = empty((2,), dtype=_F32, device=device)
    else:
        if out.dtype is not _F32 or out.shape != (2,) or not out.is_contiguous():
            raise ValueError("out must be a contiguous float32 tensor of 2")
        _same_device(dev, out=out)
    wsptr, nbytes = None, grads._workspace_bytes
    if workspace is not None:
        _same_device(dev, workspace=workspace)
        wsptr, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif nbytes:
        workspace = empty((nbytes,), dtype=torch.uint8, device=device)
        wsptr = workspace.data_ptr()
    code = _od.lib().dion_grad_norm(grads.count, table, max_norm, out.data_ptr(), wsptr, nbytes, _raw_stream(dev))
    if code == _od.DION_ERR_WORKSPACE and workspace is None:
        grads._workspace_bytes = dion_grad_norm_workspace_size(grads.count)
        return dion_grad_norm(grads, max_norm=max_norm, out=out)
    if code:
        _od._check(code, "dion_grad_norm")
    return out


def dion_adamw_step(plan, *, step, lr=None, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, grad_scale=None, seed=0,
                    hyper=None, workspace=None, stream=None):
    """One AdamW step on all tensors of a plan, in place.

    step: the number of this step, from 1.  grad_scale: a float32 CUDA tensor whose
    one value multiplies the gradients (NaN: nothing is done), as dion_grad_norm
    leaves it.  seed: of the rounding of 8-bit states.

    With `hyper`, a float64 CUDA tensor of (lr, beta1, beta2, eps, weight_decay),
    these are read on the device when the step runs, and `step` is an int64 CUDA
    tensor of one value, the number of steps taken, which the step counts up: a
    CUDA graph of the call follows both."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_adamw_step(plan, step=step, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                                   grad_scale=grad_scale, seed=seed, hyper=hyper, workspace=workspace)
    table, dev = plan._use(), plan.device
    if not isinstance(plan, AdamWPlan):
        raise TypeError("expected a plan of dion_adamw_plan")
    if dev is None:
        if hyper is None:
            return
        dev = _current_device()                    # (a step of nothing counts all the same)
    scale = None
    if grad_scale is not None:
        if grad_scale.dtype is not _F32 or grad_scale.numel() != 1:
            raise ValueError("grad_scale must be a float32 tensor of one value")
        if grad_scale.get_device() != dev:
            _same_device(dev, grad_scale=grad_scale)
        scale = grad_scale.data_ptr()
    seed &= 0xFFFFFFFF
    if hyper is None:
        if lr is None or isinstance(step, torch.Tensor):
            raise ValueError("lr and a whole number for step are required unless hyper is given")
        code = _od.lib().dion_adamw_step(plan.count, table, lr, betas[0], betas[1], eps, weight_decay, step, seed, scale,
                                         _raw_stream(dev))
    else:
        if hyper.dtype is not torch.float64 or hyper.shape != (5,) or not hyper.is_contiguous():
            raise ValueError("hyper must be a contiguous float64 tensor of (lr, beta1, beta2, eps, weight_decay)")
        if not isinstance(step, torch.Tensor) or step.dtype is not torch.int64 or step.numel() != 1:
            raise ValueError("step must be an int64 tensor of one value where hyper is given")
        if workspace is None:
            workspace = empty((256,), dtype=torch.uint8, device=step.device)
        _same_device(dev, hyper=hyper, step=step, workspace=workspace)
        code = _od.lib().dion_adamw_step_dev(plan.count, table, hyper.data_ptr(), step.data_ptr(), seed, scale,
                                             workspace.data_ptr(), workspace.numel() * workspace.element_size(), _raw_stream(dev))
    if code:
        _od._check(code, "dion_adamw_step")

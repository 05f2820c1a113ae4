"""Python binding of include/policy.h: the operators of a policy with memory.

    recurrence, recurrence_step     gated linear recurrence over [L, N, D]

`recurrence` takes part in torch's autograd; its gradient runs in the
library's kernels too.  Calls run on torch's current stream, on the current
device, where their tensors must live; outputs and workspaces come from
torch's allocator, so captured graphs keep their own.
"""
from __future__ import annotations

import ctypes as C

import torch

POLICY_F32, POLICY_BF16, POLICY_F16 = 0, 1, 2
RECUR_LINEAR, RECUR_SIGMOID = 0, 1
EXPORTED = ("recur_workspace", "recur_forward", "recur_backward", "recur_step")

_DTYPES = {torch.float32: POLICY_F32, torch.bfloat16: POLICY_BF16, torch.float16: POLICY_F16}
_FORMS = {"linear": RECUR_LINEAR, "sigmoid": RECUR_SIGMOID}


class RecurArgs(C.Structure):
    _fields_ = ([(n, C.c_int32) for n in ("steps", "rows", "width", "dtype", "form")] +
                [(n, C.c_int64) for n in ("x_step", "x_row", "gate_step", "gate_row",
                                          "h_step", "h_row")] +
                [(n, C.c_void_p) for n in ("x", "gate", "h0", "dones", "h", "h_last",
                                           "workspace")] +
                [("workspace_bytes", C.c_int64)])


class RecurGradArgs(C.Structure):
    _fields_ = ([(n, C.c_int32) for n in ("steps", "rows", "width", "dtype", "form")] +
                [(n, C.c_int64) for n in ("x_step", "x_row", "gate_step", "gate_row",
                                          "h_step", "h_row", "dh_step", "dh_row",
                                          "dx_step", "dx_row", "dgate_step", "dgate_row")] +
                [(n, C.c_void_p) for n in ("x", "gate", "h", "h0", "dones", "dh", "dh_last",
                                           "dx", "dgate", "dh0", "workspace")] +
                [("workspace_bytes", C.c_int64)])


def declare(lib):
    """Argument types of the entry points of include/policy.h."""
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    lib.recur_workspace.argtypes = [i32, i32, i32, i32]
    lib.recur_workspace.restype = i64
    lib.recur_forward.argtypes = [C.POINTER(RecurArgs), vp]
    lib.recur_backward.argtypes = [C.POINTER(RecurGradArgs), vp]
    lib.recur_step.argtypes = [i32, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp]
    for name in ("recur_forward", "recur_backward", "recur_step"):
        getattr(lib, name).restype = C.c_int


def _call(fn, *args):
    from . import _check
    _check(fn(*args))


def _lib():
    from . import load_library
    return load_library()


def _here(name, *tensors):
    """The current device's stream; every tensor must live on that device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and (not t.is_cuda or t.device.index != dev):
            raise ValueError(f"{name}: every tensor must be on the current device, cuda:{dev} "
                             f"(got {t.device})")
    return torch.cuda.current_stream().cuda_stream


def _element(name, t):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return _DTYPES[t.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _exact(name, t, dtype, shape):
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _flags(name, t, shape):
    """u8 flags; torch's truth values are u8 in memory."""
    if t is not None and t.dtype == torch.bool:
        t = t.view(torch.uint8)
    _exact(name, t, torch.uint8, shape)
    return t


def _form(form):
    if form not in _FORMS:
        raise ValueError(f"form must be 'linear' or 'sigmoid', got {form!r}")
    return _FORMS[form]


def _unit(name, t, axes):
    """Strides of all but the last axis; the last must have unit stride."""
    if t.dim() != axes:
        raise ValueError(f"{name} must have {axes} dimensions, got {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.stride()[:-1]


def _no_grad(name, *tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{name} records no gradient: call it under torch.no_grad()")


def _workspace(like, bytes_):
    return torch.empty(bytes_, dtype=torch.uint8, device=like.device) if bytes_ else None


# ---------------------------------------------------------------- recurrence
def _recur_forward(x, gate, h0, dones, form, h_last=True):
    L, N, D = x.shape
    lib, stream = _lib(), _here("recurrence", x, gate, h0, dones)
    h = torch.empty_like(x)
    last = torch.empty((N, D), dtype=torch.float32, device=x.device) if h_last else None
    a = RecurArgs(steps=L, rows=N, width=D, dtype=_DTYPES[x.dtype], form=form)
    a.x_step, a.x_row = _unit("x", x, 3)
    a.gate_step, a.gate_row = _unit("gate", gate, 3)
    a.h_step, a.h_row = h.stride()[:2]
    a.x, a.gate, a.h0, a.dones = _ptr(x), _ptr(gate), _ptr(h0), _ptr(dones)
    a.h, a.h_last = _ptr(h), _ptr(last)
    a.workspace_bytes = lib.recur_workspace(L, N, D, a.dtype)
    ws = _workspace(x, max(0, a.workspace_bytes))
    a.workspace = _ptr(ws)
    _call(lib.recur_forward, C.byref(a), stream)
    return h, last


def _recur_backward(x, gate, h, h0, dones, dh, dh_last, form, want_dh0):
    L, N, D = gate.shape
    lib, stream = _lib(), _here("recurrence", x, gate, h, h0, dones, dh, dh_last)
    dx, dgate = torch.empty_like(h), torch.empty_like(gate)
    dh0 = torch.empty((N, D), dtype=torch.float32, device=gate.device) if want_dh0 else None
    a = RecurGradArgs(steps=L, rows=N, width=D, dtype=_DTYPES[gate.dtype], form=form)
    if x is not None:
        a.x_step, a.x_row = x.stride()[:2]
    a.gate_step, a.gate_row = gate.stride()[:2]
    a.h_step, a.h_row = h.stride()[:2]
    a.dh_step, a.dh_row = dh.stride()[:2]
    a.dx_step, a.dx_row = dx.stride()[:2]
    a.dgate_step, a.dgate_row = dgate.stride()[:2]
    a.x, a.gate, a.h, a.h0, a.dones = _ptr(x), _ptr(gate), _ptr(h), _ptr(h0), _ptr(dones)
    a.dh, a.dh_last, a.dx, a.dgate, a.dh0 = _ptr(dh), _ptr(dh_last), _ptr(dx), _ptr(dgate), _ptr(dh0)
    a.workspace_bytes = lib.recur_workspace(L, N, D, a.dtype)
    ws = _workspace(gate, max(0, a.workspace_bytes))
    a.workspace = _ptr(ws)
    _call(lib.recur_backward, C.byref(a), stream)
    return dx, dgate, dh0


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, h0, dones, form):
        h, last = _recur_forward(x, gate, h0, dones, form)
        ctx.save_for_backward(x if form == RECUR_SIGMOID else None, gate, h, h0, dones)
        ctx.form = form
        ctx.set_materialize_grads(False)
        return h, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dh_last):
        x, gate, h, h0, dones = ctx.saved_tensors
        if dh is None and dh_last is None:
            return None, None, None, None, None
        dh = torch.zeros_like(h) if dh is None else dh
        if dh.shape[-1] > 1 and dh.stride(-1) != 1:
            dh = dh.contiguous()
        if dh_last is not None:
            dh_last = dh_last.contiguous()
        dx, dgate, dh0 = _recur_backward(x, gate, h, h0, dones, dh, dh_last, ctx.form,
                                         h0 is not None and ctx.needs_input_grad[2])
        return dx, dgate, dh0, None, None


def recurrence(x, gate, h0=None, dones=None, form: str = "sigmoid"):
    """Gated linear recurrence over a rollout (include/policy.h): returns
    (h, h_last).  x, gate: [L, N, D] of one dtype (float32, bfloat16,
    float16), the last dimension contiguous, the others with any strides
    (a batch-first tensor is passed transposed); h0: [N, D] float32 or None
    (zero); dones: [L, N] uint8 or bool, a collection's, or None.  h has x's
    dtype, h_last [N, D] is float32 and starts the next rollout.  Gradients
    flow to x, gate and h0."""
    f = _form(form)
    _element("x", x)
    if x.dim() != 3:
        raise ValueError(f"x must be [L, N, D], got {tuple(x.shape)}")
    if gate.dtype != x.dtype or gate.shape != x.shape:
        raise ValueError(f"gate must have x's dtype and shape, {x.dtype} {tuple(x.shape)}; got "
                         f"{gate.dtype} {tuple(gate.shape)}")
    L, N, D = x.shape
    _unit("x", x, 3)
    _unit("gate", gate, 3)
    _exact("h0", h0, torch.float32, (N, D))
    dones = _flags("dones", dones, (L, N))
    return _Recurrence.apply(x, gate, h0, dones, f)


def recurrence_step(x, gate, state, resets=None, form: str = "sigmoid", out_state=None):
    """One step for acting: returns (h, new_state).  x, gate: [N, D];
    state: [N, D] float32; resets: [N] uint8 or bool, rows whose episode ended
    before this step (their state counts as zero), or None.  out_state may
    be `state` itself, to update it in place.  It records no gradient:
    inputs that ask for one are refused unless under torch.no_grad()."""
    f = _form(form)
    _no_grad("recurrence_step", x, gate, state)
    dt = _element("x", x)
    (x_row,), (gate_row,) = _unit("x", x, 2), _unit("gate", gate, 2)
    if gate.dtype != x.dtype or gate.shape != x.shape:
        raise ValueError(f"gate must have x's dtype and shape, {x.dtype} {tuple(x.shape)}; got "
                         f"{gate.dtype} {tuple(gate.shape)}")
    N, D = x.shape
    _exact("state", state, torch.float32, (N, D))
    _exact("out_state", out_state, torch.float32, (N, D))
    resets = _flags("resets", resets, (N,))
    stream = _here("recurrence_step", x, gate, state, resets, out_state)
    h = torch.empty((N, D), dtype=x.dtype, device=x.device)
    new = torch.empty_like(state) if out_state is None else out_state
    _call(_lib().recur_step, N, D, dt, f, _ptr(x), x_row, _ptr(gate), gate_row, _ptr(state),
          _ptr(resets), _ptr(h), D, _ptr(new), stream)
    return h, new

"""Python binding of include/policy.h: the operators of a policy with memory.

    embed                           scaled embedding lookup
    recurrence, recurrence_step     gated linear recurrence over [L, N, D]
    shape_logits                    penalties, bias and mask on logits

`embed`, `recurrence` and `shape_logits` take part in torch's autograd; their
gradients run in the library's kernels too.  Forward-mode derivatives and the
transforms of torch.func are refused.  Calls run on torch's current
stream, on the current device, where their tensors must live; outputs and
workspaces come from torch's allocator, so captured graphs keep their own.

A backward pass that is captured into a graph asks for its gradients with
torch.autograd.grad, or is captured when no eager graph of the same leaves is
alive: torch accumulates into a leaf's .grad on the stream on which the leaf was
first used, and to wait for that stream inside a capture ends the process.
"""
from __future__ import annotations

import ctypes as C

import torch
import torch.autograd.forward_ad as _forward_ad

POLICY_F32, POLICY_BF16, POLICY_F16 = 0, 1, 2
RECUR_LINEAR, RECUR_SIGMOID = 0, 1
LOGITS_MASK_NONE, LOGITS_MASK_BYTES, LOGITS_MASK_BITS = 0, 1, 2
EXPORTED = ("recur_workspace", "recur_kept_workspace", "recur_forward", "recur_backward",
            "recur_forward_kept", "recur_backward_kept", "recur_step",
            "embed_forward", "embed_workspace", "embed_backward",
            "logits_forward", "logits_workspace", "logits_backward")

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


class LogitsArgs(C.Structure):
    _fields_ = [("rows", C.c_int64), ("vocab", C.c_int32), ("dtype", C.c_int32),
                ("logits", C.c_void_p), ("logits_row", C.c_int64),
                ("bias", C.c_void_p), ("bias_row", C.c_int64),
                ("history", C.c_void_p), ("history_row", C.c_int64),
                ("history_len", C.c_void_p), ("history_width", C.c_int32),
                ("mask_kind", C.c_int32),
                ("repetition", C.c_float), ("presence", C.c_float), ("frequency", C.c_float),
                ("repetition_rows", C.c_void_p), ("presence_rows", C.c_void_p),
                ("frequency_rows", C.c_void_p),
                ("mask", C.c_void_p), ("mask_row", C.c_int64), ("mask_count", C.c_int64),
                ("mask_rows", C.c_void_p)]


def declare(lib):
    """Argument types of the entry points of include/policy.h."""
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    lib.recur_workspace.argtypes = lib.recur_kept_workspace.argtypes = [i32, i32, i32, i32]
    lib.recur_forward.argtypes = [C.POINTER(RecurArgs), vp]
    lib.recur_backward.argtypes = [C.POINTER(RecurGradArgs), vp]
    lib.recur_forward_kept.argtypes = [C.POINTER(RecurArgs), vp, vp]
    lib.recur_backward_kept.argtypes = [C.POINTER(RecurGradArgs), vp, vp]
    lib.recur_step.argtypes = [i32, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp]
    lib.embed_forward.argtypes = [i32, vp, i64, i32, i64, vp, i32, i64, C.c_float, vp, i64, vp]
    lib.embed_workspace.argtypes = [i32, i64, i32, i64]
    lib.embed_backward.argtypes = [i32, vp, i64, vp, i32, i64, i64, i32, C.c_float, vp, i64, vp,
                                   i64, vp]
    lib.logits_forward.argtypes = [C.POINTER(LogitsArgs), vp, i64, vp]
    lib.logits_workspace.argtypes = [i64, i32]
    lib.logits_backward.argtypes = [C.POINTER(LogitsArgs), vp, i64, vp, i64, vp, vp, i64, vp]
    for name in EXPORTED:
        getattr(lib, name).restype = i64 if name.endswith("_workspace") else C.c_int


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import load_library
        _loaded = load_library()
    return _loaded


def _call(fn, *args):
    rc = fn(*args)
    if rc != 0:
        from . import _check
        _check(rc)


# the raw stream handle without building a stream object, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(name, *tensors):
    """The current device's stream; every tensor must live on that device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: every tensor must be on the current device, cuda:{dev} "
                             f"(got {t.device})")
    return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream().cuda_stream


def _there(t):
    """The stream of a backward pass: it runs on the device of its gradients,
    where the forward call's tensors are known to live."""
    return _raw_stream(t.get_device()) if _raw_stream else torch.cuda.current_stream().cuda_stream


def _first_order(backward):
    """A backward pass whose results have no gradient.  torch's own guard for
    that costs a third of a small pass's time on the host, and is needed only
    where a graph over the gradients is asked for."""
    guarded = torch.autograd.function.once_differentiable(backward)

    def run(ctx, *grads):
        if _forward_ad._current_level >= 0:
            _no_tangent("a backward pass", *grads)
        return (guarded if torch.is_grad_enabled() else backward)(ctx, *grads)
    return staticmethod(run)


def _element(name, t):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return _DTYPES[t.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _exact(name, t, dtype, shape):
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
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


def _wants_grad(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _no_grad(name, *tensors):
    if _wants_grad(*tensors):
        raise ValueError(f"{name} records no gradient: call it under torch.no_grad()")


def _no_tangent(name, *tensors):
    """Refuses a forward-mode derivative: a dual tensor asks for no gradient,
    and its tangent would be dropped without a word.  Called only where a level
    of them is open, which costs a small call less than asking here."""
    for t in tensors:
        if isinstance(t, torch.Tensor) and _forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{name} has no forward-mode derivative")


def _written(t):
    """Tells autograd that the caller's tensor has new values, so that a graph
    which saved the old ones raises instead of using these."""
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _apart_or_same(name, out, t):
    """The output is the input itself, or shares no element with it.  Both have
    the same type and rows of the same width, given apart by their strides."""
    shift = (out.data_ptr() - t.data_ptr()) // t.element_size()
    width, rows = t.shape[-1], t.numel() // t.shape[-1] if t.shape[-1] else 0
    if rows == 0:
        return
    strides = [width if u.is_contiguous() else u.stride(0) for u in (t, out)]
    if (shift == 0 and (rows == 1 or strides[0] == strides[1])) or \
            shift >= (rows - 1) * strides[0] + width or -shift >= (rows - 1) * strides[1] + width:
        return
    # interleaved rows of one buffer: every row lies between two of the other's
    if strides[0] == strides[1]:
        shared = not width <= shift % strides[0] <= strides[0] - width
    else:
        a, b = torch.arange(rows) * strides[0], torch.arange(rows) * strides[1] + shift
        k = torch.searchsorted(a, b)
        shared = bool(((b - a[(k - 1).clamp(min=0)] < width) & (k > 0) |
                       (a[k.clamp(max=rows - 1)] - b < width) & (k < rows)).any())
    if not shared:
        return
    raise ValueError(f"{name} must be the input itself or not overlap it")


def _workspace(like, bytes_):
    return torch.empty(bytes_, dtype=torch.uint8, device=like.device) if bytes_ else None


def _like(t):
    """An empty tensor of t's shape, in its layout where that leaves the last
    dimension contiguous (of overlapping windows torch derives one that does not)."""
    e = torch.empty_like(t)
    if t.shape[-1] > 1 and e.stride(-1) != 1:
        e = torch.empty(t.shape, dtype=t.dtype, device=t.device)
    return e


# ---------------------------------------------------------------- recurrence
def _recur_forward(x, gate, h0, dones, form, kept=None):
    L, N, D = x.shape
    lib, stream = _lib(), _here("recurrence", x, gate, h0, dones)
    h = _like(x)
    last = torch.empty((N, D), dtype=torch.float32, device=x.device)
    dt = _DTYPES[x.dtype]
    size = lib.recur_kept_workspace(L, N, D, dt)
    ws = _workspace(x, size)
    a = RecurArgs(L, N, D, dt, form, *x.stride()[:2], *gate.stride()[:2], *h.stride()[:2],
                  _ptr(x), _ptr(gate), _ptr(h0), _ptr(dones), _ptr(h), _ptr(last), _ptr(ws), size)
    if kept is None:
        _call(lib.recur_forward, C.byref(a), stream)
    else:
        _call(lib.recur_forward_kept, C.byref(a), _ptr(kept), stream)
    return h, last


def _recur_backward(x, gate, h, kept, h0, dones, dh, dh_last, form, want_dh0):
    L, N, D = gate.shape
    lib, stream = _lib(), _there(dh)
    dx, dgate = _like(x if h is None else h), _like(gate)
    dh0 = torch.empty((N, D), dtype=torch.float32, device=gate.device) if want_dh0 else None
    dt = _DTYPES[gate.dtype]
    size = lib.recur_kept_workspace(L, N, D, dt)
    ws = _workspace(gate, size)
    a = RecurGradArgs(L, N, D, dt, form, *(x.stride()[:2] if x is not None else (0, 0)),
                      *gate.stride()[:2], *(h.stride()[:2] if h is not None else (0, 0)),
                      *dh.stride()[:2], *dx.stride()[:2], *dgate.stride()[:2],
                      _ptr(x), _ptr(gate), _ptr(h), _ptr(h0), _ptr(dones), _ptr(dh), _ptr(dh_last), _ptr(dx), _ptr(dgate), _ptr(dh0), _ptr(ws), size)
    _call(lib.recur_backward_kept, C.byref(a), _ptr(kept), stream)
    return dx, dgate, dh0


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, h0, dones, form):
        # the gradient takes the states of 16-bit sigmoid gates from `kept`, not from h
        kept = None
        if form == RECUR_SIGMOID and x.dtype != torch.float32:
            kept = torch.empty(((x.shape[0] + 7) // 8,) + x.shape[1:], dtype=torch.float32, device=x.device)
        h, last = _recur_forward(x, gate, h0, dones, form, kept)
        ctx.save_for_backward(x if form == RECUR_SIGMOID else None, gate, h if kept is None else None, kept,
                              h0, dones)
        ctx.form = form
        ctx.set_materialize_grads(False)
        return h, last

    @_first_order
    def backward(ctx, dh, dh_last):
        x, gate, h, kept, h0, dones = ctx.saved_tensors
        if dh is None and dh_last is None:
            return None, None, None, None, None
        dh = torch.zeros(gate.shape, dtype=gate.dtype, device=gate.device) if dh is None else dh
        if dh.shape[-1] > 1 and dh.stride(-1) != 1:
            dh = dh.contiguous()
        if dh_last is not None:
            dh_last = dh_last.contiguous()
        dx, dgate, dh0 = _recur_backward(x, gate, h, kept, h0, dones, dh, dh_last, ctx.form,
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
    if _forward_ad._current_level >= 0:
        _no_tangent("recurrence", x, gate, h0)
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
    if not _wants_grad(x, gate, h0):
        return _recur_forward(x, gate, h0, dones, f)
    return _Recurrence.apply(x, gate, h0, dones, f)


def recurrence_step(x, gate, state, resets=None, form: str = "sigmoid", out_state=None):
    """One step for acting: returns (h, new_state).  x, gate: [N, D];
    state: [N, D] float32; resets: [N] uint8 or bool, rows whose episode ended
    before this step (their state counts as zero), or None.  out_state may
    be `state` itself, to update it in place.  It records no gradient:
    inputs that ask for one are refused unless under torch.no_grad()."""
    f = _form(form)
    if _forward_ad._current_level >= 0:
        _no_tangent("recurrence_step", x, gate, state, out_state)
    _no_grad("recurrence_step", x, gate, state, out_state)
    dt = _element("x", x)
    (x_row,), (gate_row,) = _unit("x", x, 2), _unit("gate", gate, 2)
    if gate.dtype != x.dtype or gate.shape != x.shape:
        raise ValueError(f"gate must have x's dtype and shape, {x.dtype} {tuple(x.shape)}; got "
                         f"{gate.dtype} {tuple(gate.shape)}")
    N, D = x.shape
    _exact("state", state, torch.float32, (N, D))
    _exact("out_state", out_state, torch.float32, (N, D))
    if out_state is not None:
        _apart_or_same("out_state", out_state, state)
    resets = _flags("resets", resets, (N,))
    stream = _here("recurrence_step", x, gate, state, resets, out_state)
    h = torch.empty((N, D), dtype=x.dtype, device=x.device)
    new = torch.empty_like(state) if out_state is None else out_state
    _call(_lib().recur_step, N, D, dt, f, _ptr(x), x_row, _ptr(gate), gate_row, _ptr(state),
          _ptr(resets), _ptr(h), D, _ptr(new), stream)
    if out_state is not None:
        _written(out_state)
    return h, new


# ----------------------------------------------------------------- embedding
_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}


def _embed_forward(weight, index, scale):
    V, D = weight.shape
    stream = _here("embed", weight, index)
    out = torch.empty(index.shape + (D,), dtype=weight.dtype, device=weight.device)
    _call(_lib().embed_forward, _DTYPES[weight.dtype], _ptr(weight), V, D, max(D, weight.stride(0)),
          _ptr(index), _INDEX_BYTES[index.dtype], index.numel(), scale, _ptr(out), D, stream)
    return out


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, index, scale):
        ctx.save_for_backward(index)
        V, D = weight.shape
        dt, count = _DTYPES[weight.dtype], index.numel()
        ctx.sizes = V, D, dt, count, scale, _lib().embed_workspace(dt, V, D, count)
        return _embed_forward(weight, index, scale)

    @_first_order
    def backward(ctx, dout):
        index, = ctx.saved_tensors
        V, D, dt, count, scale, size = ctx.sizes
        if not dout.is_contiguous():
            dout = dout.contiguous()
        dweight = dout.new_empty((V, D))
        ws = _workspace(dout, size)
        _call(_lib().embed_backward, dt, dout.data_ptr(), D, index.data_ptr(),
              _INDEX_BYTES[index.dtype], count, V, D, scale, dweight.data_ptr(), D, _ptr(ws), size,
              _there(dout))
        return dweight, None, None


def embed(weight, index, scale: float = 1.0):
    """scale * weight[index] (include/policy.h): weight [V, D] float32, bfloat16
    or float16 with contiguous rows, index a contiguous int32 or int64 tensor
    of any shape; returns index.shape + [D] in weight's dtype.  An index outside
    [0, V), such as the -1 of an episode's first step, gives zeros.  The
    gradient flows to weight and is dense."""
    if _forward_ad._current_level >= 0:
        _no_tangent("embed", weight)
    _element("weight", weight)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [V, D], got {tuple(weight.shape)}")
    _unit("weight", weight, 2)
    if weight.shape[0] > 1 and weight.stride(0) < weight.shape[1]:
        raise ValueError("weight's rows must not overlap")
    if index.dtype not in _INDEX_BYTES:
        raise ValueError(f"index must be int32 or int64, got {index.dtype}")
    if not index.is_contiguous():
        raise ValueError("index must be contiguous")
    if not _wants_grad(weight):
        return _embed_forward(weight, index, float(scale))
    return _Embed.apply(weight, index, float(scale))


# -------------------------------------------------------------------- logits
def _logits_args(logits, bias, history, history_len, penalties, mask, mask_rows):
    """The C struct; every tensor has been checked.  penalties: repetition,
    presence, frequency, each a number or a tensor."""
    V = logits.shape[-1]
    row = logits.stride(0) if logits.dim() == 2 and logits.shape[0] > 1 else V
    H = 0 if history is None else history.shape[-1]
    scalars, rows = [1.0, 0.0, 0.0], [None, None, None]
    for i, p in enumerate(penalties):
        if isinstance(p, torch.Tensor):
            rows[i] = p.data_ptr()
        else:
            scalars[i] = p
    kind, mask_row, mask_count = LOGITS_MASK_NONE, 0, 0
    if mask is not None:
        kind = LOGITS_MASK_BITS if mask.dtype is torch.int32 else LOGITS_MASK_BYTES
        mask_row = mask.shape[-1]
        mask_count = mask.numel() // mask_row if mask_row else 0
    return LogitsArgs(logits.numel() // V if V else 0, V, _DTYPES[logits.dtype], _ptr(logits), row,
                      _ptr(bias), V if bias is not None and bias.dim() > 1 else 0, _ptr(history), H,
                      _ptr(history_len), H, kind, *scalars, *rows, _ptr(mask), mask_row, mask_count,
                      _ptr(mask_rows))


def _logits_forward(logits, bias, history, history_len, penalties, mask, mask_rows, out):
    stream = _here("shape_logits", logits, bias, history, history_len, mask, mask_rows, out,
                   *[p for p in penalties if isinstance(p, torch.Tensor)])
    a = _logits_args(logits, bias, history, history_len, penalties, mask, mask_rows)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    out_row = out.stride(0) if out.dim() == 2 and out.shape[0] > 1 else a.vocab
    _call(_lib().logits_forward, C.byref(a), _ptr(out), out_row, stream)
    return out


class _ShapeLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, history, history_len, penalties, mask, mask_rows):
        out = _logits_forward(logits, bias, history, history_len, penalties, mask, mask_rows, None)
        # of the penalties only the repetition scales the gradient
        rep = penalties[0]
        ctx.repetition = None if isinstance(rep, torch.Tensor) else rep
        if history is None or ctx.repetition == 1.0:
            logits, history, history_len = None, None, None
        ctx.save_for_backward(logits, history, history_len, mask, mask_rows,
                              rep if ctx.repetition is None else None)
        return out

    @_first_order
    def backward(ctx, dout):
        logits, history, history_len, mask, mask_rows, rep = ctx.saved_tensors
        lib, stream = _lib(), _there(dout)
        V = dout.shape[-1]
        dout = dout.contiguous()
        a = _logits_args(dout if logits is None else logits, None, history, history_len,
                         (ctx.repetition if rep is None else rep,), mask, mask_rows)
        dlogits = torch.empty_like(dout) if ctx.needs_input_grad[0] else None
        dbias = torch.empty(V, dtype=torch.float32, device=dout.device) \
            if ctx.needs_input_grad[1] else None
        size = lib.logits_workspace(a.rows, V) if dbias is not None else 0
        ws = _workspace(dout, size)
        _call(lib.logits_backward, C.byref(a), _ptr(dout), V, _ptr(dlogits), V, _ptr(dbias), _ptr(ws),
              size, stream)
        return dlogits, dbias, None, None, None, None, None


def _per_row(name, value, lead):
    if isinstance(value, torch.Tensor):
        _exact(name, value, torch.float32, lead)
        if _wants_grad(value):
            raise ValueError(f"{name} takes no gradient")
        return value
    return float(value)


def shape_logits(logits, bias=None, history=None, history_len=None, repetition=1.0, presence=0.0,
                 frequency=0.0, mask=None, mask_rows=None, out=None):
    """Penalties for tokens of the history, then the bias, then the mask
    (include/policy.h); returns a tensor like `logits`, -inf where masked.

    logits: [..., V] float32, bfloat16 or float16, contiguous (or [R, V] with
    contiguous rows).  bias: [V] or logits' shape, float32.  history: [..., H]
    int32 token ids (others, such as a padding of -1, are ignored), of which
    the first history_len [...] int32 count.  repetition, presence and
    frequency: a number or one float32 per row [...].  mask: uint8 or bool
    [..., V], or int32 [..., ceil(V / 32)] with token v at bit v % 32 of word
    v // 32; one row per row of logits, a single row for all, or any number of
    rows chosen by mask_rows [...] int32 (a value that names no row allows
    everything).  out: written instead of a new tensor; may be `logits`, else
    it must not overlap it.
    Gradients flow to logits and to a bias of shape [V]."""
    if _forward_ad._current_level >= 0:
        _no_tangent("shape_logits", logits, bias, repetition, presence, frequency, out)
    _element("logits", logits)
    if logits.dim() < 1:
        raise ValueError("logits must be [..., V]")
    V, lead = logits.shape[-1], logits.shape[:-1]
    if not logits.is_contiguous():
        _unit("logits", logits, 2)
        if logits.stride(0) < V:
            raise ValueError("logits' rows must not overlap")
    if bias is not None:
        _exact("bias", bias, torch.float32, (V,) if bias.dim() == 1 else lead + (V,))
        if bias.dim() > 1 and _wants_grad(bias):
            raise ValueError("only a bias of shape [V] takes a gradient")
    if history is not None:
        H = history.shape[-1] if history.dim() else 0
        _exact("history", history, torch.int32, lead + (H,))
        _exact("history_len", history_len, torch.int32, lead)
    elif history_len is not None:
        raise ValueError("history_len needs a history")
    penalties = (_per_row("repetition", repetition, lead), _per_row("presence", presence, lead),
                 _per_row("frequency", frequency, lead))
    if mask is not None:
        if mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        if mask.dtype not in (torch.uint8, torch.int32):
            raise ValueError(f"mask must be uint8, bool or int32, got {mask.dtype}")
        width = (V + 31) // 32 if mask.dtype == torch.int32 else V
        if mask.dim() < 1 or mask.shape[-1] != width:
            raise ValueError(f"mask's last dimension must be {width}, got shape {tuple(mask.shape)}")
        if not mask.is_contiguous():
            raise ValueError("mask must be contiguous")
        if mask_rows is not None:
            _exact("mask_rows", mask_rows, torch.int32, lead)
        elif mask.numel() != width and mask.shape[:-1] != lead:
            raise ValueError(f"mask must have one row or rows {tuple(lead)}, got shape {tuple(mask.shape)}")
    elif mask_rows is not None:
        raise ValueError("mask_rows needs a mask")
    if out is not None:
        _no_grad("shape_logits with out", logits, bias, out)
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out must have logits' dtype and shape")
        if not out.is_contiguous():
            _unit("out", out, 2)
            if out.stride(0) < V:
                raise ValueError("out's rows must not overlap")
        _apart_or_same("out", out, logits)
    if out is not None or not _wants_grad(logits, bias):
        result = _logits_forward(logits, bias, history, history_len, penalties, mask, mask_rows, out)
        if out is not None:
            _written(out)
        return result
    return _ShapeLogits.apply(logits, bias, history, history_len, penalties, mask, mask_rows)

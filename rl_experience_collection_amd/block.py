"""Python binding of include/block.h: the operators of a residual block with a
selective memory, over [L, N, D] rollouts.

    causal_conv, causal_conv_step         short causal convolution
    selective_scan, selective_scan_step   selective state space scan
    residual_norm                         norms around a block, gate, residual, dropout
    dropout                               dropout from a counter, no mask stored

`causal_conv`, `selective_scan`, `residual_norm` and `dropout` take part in
torch's autograd; their gradients run in the library's kernels too.  Streams,
devices, workspaces, captured graphs and refused derivatives are those of
policy.py.
"""
from __future__ import annotations

import ctypes as C
import math
import struct

import torch

from .policy import (_DTYPES, _apart_or_same, _call, _element, _exact, _first_order, _flags,
                     _forward_ad, _here, _lib, _like, _no_grad, _no_tangent, _ptr, _there, _unit,
                     _wants_grad, _workspace, _written)

BLOCK_NONE, BLOCK_SIGMOID, BLOCK_SILU = 0, 1, 2
EXPORTED = ("conv_forward", "conv_workspace", "conv_backward", "conv_step",
            "scan_kept", "scan_workspace", "scan_grad_workspace", "scan_forward", "scan_backward", "scan_step",
            "norm_forward", "norm_workspace", "norm_backward", "drop_forward")

_ACTIVATIONS = {"none": BLOCK_NONE, "sigmoid": BLOCK_SIGMOID, "silu": BLOCK_SILU}
_f32 = torch.float32


def _fields(kind, names):
    return [(n, kind) for n in names.split()]


class ConvArgs(C.Structure):
    _fields_ = (_fields(C.c_int32, "steps rows width taps dtype activation") +
                _fields(C.c_int64, "x_step x_row y_step y_row") +
                _fields(C.c_void_p, "x weight bias state dones y new_state"))


class ConvGradArgs(C.Structure):
    _fields_ = ([("f", ConvArgs)] + _fields(C.c_int64, "dy_step dy_row dx_step dx_row") +
                _fields(C.c_void_p, "dy dnew_state dx dweight dbias dstate workspace") +
                [("workspace_bytes", C.c_int64)])


class ScanArgs(C.Structure):
    _fields_ = (_fields(C.c_int32, "steps rows width states groups dtype softplus") +
                _fields(C.c_int64, "x_step x_row delta_step delta_row gate_step gate_row b_step b_row "
                                   "b_group c_step c_row c_group y_step y_row") +
                _fields(C.c_void_p, "x delta gate b c rate skip delta_bias state dones y new_state kept "
                                    "workspace") +
                [("workspace_bytes", C.c_int64)])


class ScanGradArgs(C.Structure):
    _fields_ = ([("f", ScanArgs)] +
                _fields(C.c_int64, "dy_step dy_row dx_step dx_row ddelta_step ddelta_row dgate_step "
                                   "dgate_row db_step db_row db_group dc_step dc_row dc_group") +
                _fields(C.c_void_p, "dy dnew_state dx ddelta dgate db dc drate dskip ddelta_bias dstate"))


class NormArgs(C.Structure):
    _fields_ = ([("rows", C.c_int64)] + _fields(C.c_int32, "width dtype branch_norm activation") +
                _fields(C.c_float, "residual_scale branch_scale eps drop") +
                [("seed", C.c_uint64), ("seed_at", C.c_void_p), ("offset", C.c_uint32), ("pad", C.c_uint32),
                 ("residual", C.c_void_p), ("residual_row", C.c_int64), ("branch", C.c_void_p),
                 ("branch_row", C.c_int64), ("gate", C.c_void_p), ("gate_row", C.c_int64),
                 ("weight", C.c_void_p), ("branch_weight", C.c_void_p)])


class NormGradArgs(C.Structure):
    _fields_ = ([("f", NormArgs), ("stats", C.c_void_p), ("dstream", C.c_void_p), ("dstream_row", C.c_int64),
                 ("dnormed", C.c_void_p), ("dnormed_row", C.c_int64)] +
                _fields(C.c_void_p, "dresidual dbranch dgate dweight dbranch_weight workspace") +
                [("workspace_bytes", C.c_int64)])


# The same structs as bytes: packing one takes a fraction of what filling a
# ctypes structure of some forty fields does.
_CONV = struct.Struct("6i4q7Q").pack
_CONV_GRAD = struct.Struct("4q7Qq").pack
_SCAN = struct.Struct("7i4x14q14Qq").pack
_SCAN_GRAD = struct.Struct("14q11Q").pack
_NORM = struct.Struct("q4i4fQQIIQqQqQq2Q").pack
_NORM_GRAD = struct.Struct("QQqQq6Qq").pack
_packed = {}  # entry points that take them


def _at(t):
    return 0 if t is None else t.data_ptr()


def _entry(name):
    fn = _packed.get(name)
    if fn is None:
        lib = _lib()
        fn = lib[name]
        fn.argtypes, fn.restype = [C.c_char_p] + list(getattr(lib, name).argtypes[1:]), C.c_int
        _packed[name] = fn  # last: another thread may call what it finds here
    return fn


def declare(lib):
    """Argument types of the entry points of include/block.h."""
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    lib.conv_forward.argtypes = [C.POINTER(ConvArgs), vp]
    lib.conv_workspace.argtypes = [i32] * 5
    lib.conv_backward.argtypes = [C.POINTER(ConvGradArgs), vp]
    lib.conv_step.argtypes = [i32] * 5 + [vp, i64, vp, vp, vp, vp, vp, i64, vp, vp]
    lib.scan_kept.argtypes = lib.scan_workspace.argtypes = lib.scan_grad_workspace.argtypes = [i32] * 5
    lib.scan_forward.argtypes = lib.scan_step.argtypes = [C.POINTER(ScanArgs), vp]
    lib.scan_backward.argtypes = [C.POINTER(ScanGradArgs), vp]
    lib.norm_forward.argtypes = [C.POINTER(NormArgs), vp, i64, vp, i64, vp, vp]
    lib.norm_workspace.argtypes = [i64, i32, i32]
    lib.norm_backward.argtypes = [C.POINTER(NormGradArgs), vp]
    lib.drop_forward.argtypes = [i32, vp, i64, C.c_float, C.c_uint64, vp, C.c_uint32, vp, vp]
    for name in EXPORTED:
        getattr(lib, name).restype = i64 if name.endswith(("_workspace", "_kept")) else C.c_int


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation must be one of {', '.join(allowed)}, got {name!r}")
    return _ACTIVATIONS[name]


def _same(name, t, like, what):
    if t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError(f"{name} must have {what}'s dtype and shape, {like.dtype} {tuple(like.shape)}; got "
                         f"{t.dtype} {tuple(t.shape)}")


def _sizes(*sizes):
    """The library's sizes are 32-bit; its own limits are below."""
    if max(sizes) >> 31:
        raise ValueError(f"sizes must be below 2^31, got {sizes}")


def _rows_of(g):
    """A gradient whose last dimension is contiguous."""
    return g.contiguous() if g.shape[-1] > 1 and g.stride(-1) != 1 else g


# --------------------------------------------------------------- convolution
def _conv_args(x, y, weight, bias, state, dones, new_state, act):
    L, N, D = x.shape
    return _CONV(L, N, D, weight.shape[1], _DTYPES[x.dtype], act, *x.stride()[:2], *y.stride()[:2], x.data_ptr(),
                 weight.data_ptr(), _at(bias), _at(state), _at(dones), y.data_ptr(), _at(new_state))


def _conv_forward(x, weight, bias, state, dones, act):
    stream = _here("causal_conv", x, weight, bias, state, dones)
    y = _like(x)
    new = torch.empty((x.shape[1], weight.shape[1] - 1, x.shape[2]), dtype=x.dtype, device=x.device)
    _call(_entry("conv_forward"), _conv_args(x, y, weight, bias, state, dones, new, act), stream)
    return y, new


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, dones, act):
        y, new = _conv_forward(x, weight, bias, state, dones, act)
        ctx.save_for_backward(x, weight, bias, state, dones)
        ctx.act = act
        ctx.set_materialize_grads(False)
        return y, new

    @_first_order
    def backward(ctx, dy, dnew):
        x, weight, bias, state, dones = ctx.saved_tensors
        if dy is None and dnew is None:
            return (None,) * 6
        lib, stream = _lib(), _there(x)
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _rows_of(dy)
        if dnew is not None:
            dnew = dnew.contiguous()
        dx, dweight = _like(x), torch.empty_like(weight)
        dbias = torch.empty_like(bias) if bias is not None and ctx.needs_input_grad[2] else None
        dstate = torch.empty_like(state) if state is not None and ctx.needs_input_grad[3] else None
        f = _conv_args(x, x, weight, bias, state, dones, None, ctx.act)
        size = lib.conv_workspace(*x.shape, weight.shape[1], _DTYPES[x.dtype])
        ws = _workspace(x, size)
        g = f + _CONV_GRAD(*dy.stride()[:2], *dx.stride()[:2], dy.data_ptr(), _at(dnew), dx.data_ptr(),
                           dweight.data_ptr(), _at(dbias), _at(dstate), _at(ws), size)
        _call(_entry("conv_backward"), g, stream)
        return dx, dweight, dbias, dstate, None, None


def _conv_weights(x, weight, bias):
    D = x.shape[-1]
    _sizes(*x.shape)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [D, W], got {tuple(weight.shape)}")
    _exact("weight", weight, _f32, (D, weight.shape[1]))
    if not 1 <= weight.shape[1] <= 8:
        raise ValueError(f"weight must have 1 to 8 taps, got {weight.shape[1]}")
    _exact("bias", bias, _f32, (D,))
    return weight.shape[1]


def causal_conv(x, weight, bias=None, state=None, dones=None, activation: str = "silu"):
    """Short causal convolution of each channel over a rollout
    (include/block.h): returns (y, new_state).  x: [L, N, D] float32, bfloat16
    or float16, the last dimension contiguous, the others with any strides (a
    batch-first tensor is passed transposed); weight: [D, W] float32, W of 1 to
    8, the current step's tap last; bias: [D] float32; state: [N, W - 1, D] of
    x's dtype, the inputs before the first step, oldest first, or None (zero);
    dones: [L, N] uint8 or bool, a collection's: an input of a finished
    episode does not reach the next one; activation: "silu" or "none".
    new_state starts the next rollout.  Gradients flow to x, weight, bias and
    state."""
    act = _activation(activation, ("silu", "none"))
    if _forward_ad._current_level >= 0:
        _no_tangent("causal_conv", x, weight, bias, state)
    _element("x", x)
    _unit("x", x, 3)
    L, N, D = x.shape
    W = _conv_weights(x, weight, bias)
    _exact("state", state, x.dtype, (N, W - 1, D))
    dones = _flags("dones", dones, (L, N))
    if not _wants_grad(x, weight, bias, state):
        return _conv_forward(x, weight, bias, state, dones, act)
    return _CausalConv.apply(x, weight, bias, state, dones, act)


def causal_conv_step(x, weight, state, bias=None, resets=None, activation: str = "silu", out_state=None):
    """One step for acting: returns (y, new_state).  x: [N, D]; state:
    [N, W - 1, D] of x's dtype; resets: [N] uint8 or bool, rows whose episode
    ended before this step (their state counts as zero), or None.  out_state
    may be `state` itself, to update it in place.  It records no gradient."""
    act = _activation(activation, ("silu", "none"))
    if _forward_ad._current_level >= 0:
        _no_tangent("causal_conv_step", x, weight, bias, state, out_state)
    _no_grad("causal_conv_step", x, weight, bias, state, out_state)
    dt = _element("x", x)
    (x_row,) = _unit("x", x, 2)
    N, D = x.shape
    W = _conv_weights(x, weight, bias)
    _exact("state", state, x.dtype, (N, W - 1, D))
    _exact("out_state", out_state, x.dtype, (N, W - 1, D))
    if out_state is not None:
        _apart_or_same("out_state", out_state, state)
    resets = _flags("resets", resets, (N,))
    stream = _here("causal_conv_step", x, weight, state, bias, resets, out_state)
    y = x.new_empty((N, D))
    new = torch.empty_like(state) if out_state is None else out_state
    _call(_lib().conv_step, N, D, W, dt, act, _ptr(x), x_row, _ptr(weight), _ptr(bias), _ptr(state), _ptr(resets),
          _ptr(y), D, _ptr(new), stream)
    if out_state is not None:
        _written(out_state)
    return y, new


# ---------------------------------------------------------------------- scan
def _strides(t, lead):
    """Strides of the steps, rows and groups of b, c or their gradients."""
    s = t.stride()
    return s[:lead + 1] if t.dim() == lead + 2 else s[:lead] + (0,)


def _scan_args(x, delta, rate, b, c, skip, gate, delta_bias, state, dones, softplus, y, new, kept, ws, size):
    L, N, D = x.shape
    G = b.shape[2] if b.dim() == 4 else 1
    return _SCAN(L, N, D, rate.shape[1], G, _DTYPES[x.dtype], softplus, *x.stride()[:2], *delta.stride()[:2],
                 *(gate.stride()[:2] if gate is not None else (0, 0)), *_strides(b, 2), *_strides(c, 2),
                 *y.stride()[:2], x.data_ptr(), delta.data_ptr(), _at(gate), b.data_ptr(), c.data_ptr(),
                 rate.data_ptr(), _at(skip), _at(delta_bias), _at(state), _at(dones), y.data_ptr(), _at(new),
                 _at(kept), _at(ws), size)


def _scan_sizes(x, rate, b):
    return x.shape + (rate.shape[1], b.shape[2] if b.dim() == 4 else 1)


def _scan_forward(x, delta, rate, b, c, skip, gate, delta_bias, state, dones, softplus, kept=None):
    stream = _here("selective_scan", x, delta, rate, b, c, skip, gate, delta_bias, state, dones)
    y = _like(x)
    new = rate.new_empty((x.shape[1],) + rate.shape)
    size = _lib().scan_workspace(*_scan_sizes(x, rate, b))
    ws = _workspace(x, max(size, 0))
    _call(_entry("scan_forward"), _scan_args(x, delta, rate, b, c, skip, gate, delta_bias, state, dones, softplus, y,
                                             new, kept, ws, size), stream)
    return y, new


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, delta, rate, b, c, skip, gate, delta_bias, state, dones, softplus):
        # the states that the gradient starts from, one of eight
        kept = rate.new_empty(max(_lib().scan_kept(*_scan_sizes(x, rate, b)), 0))
        y, new = _scan_forward(x, delta, rate, b, c, skip, gate, delta_bias, state, dones, softplus, kept)
        ctx.save_for_backward(x, delta, rate, b, c, skip, gate, delta_bias, dones, kept)
        ctx.softplus = softplus
        ctx.has_state = state is not None
        ctx.set_materialize_grads(False)
        return y, new

    @_first_order
    def backward(ctx, dy, dnew):
        x, delta, rate, b, c, skip, gate, delta_bias, dones, kept = ctx.saved_tensors
        if dy is None and dnew is None:
            return (None,) * 11
        lib, stream = _lib(), _there(x)
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _rows_of(dy)
        if dnew is not None:
            dnew = dnew.contiguous()
        dx, ddelta, db, dc, drate = _like(x), _like(delta), _like(b), _like(c), torch.empty_like(rate)
        if x.shape[2] == 0:  # sums over no channels, which the library does not write
            db.zero_(), dc.zero_()
        dgate = _like(gate) if gate is not None else None
        needs = ctx.needs_input_grad
        dskip = torch.empty_like(skip) if skip is not None and needs[5] else None
        dbias = torch.empty_like(delta_bias) if delta_bias is not None and needs[7] else None
        dstate = None
        if ctx.has_state and needs[8]:
            dstate = rate.new_empty((x.shape[1],) + rate.shape)
        size = lib.scan_grad_workspace(*_scan_sizes(x, rate, b))
        ws = _workspace(x, size)
        f = _scan_args(x, delta, rate, b, c, skip, gate, delta_bias, None, dones, ctx.softplus, x, None, kept, ws, size)
        g = f + _SCAN_GRAD(*dy.stride()[:2], *dx.stride()[:2], *ddelta.stride()[:2],
                           *(dgate.stride()[:2] if dgate is not None else (0, 0)), *_strides(db, 2),
                           *_strides(dc, 2), dy.data_ptr(), _at(dnew), dx.data_ptr(), ddelta.data_ptr(), _at(dgate),
                           db.data_ptr(), dc.data_ptr(), drate.data_ptr(), _at(dskip), _at(dbias), _at(dstate))
        _call(_entry("scan_backward"), g, stream)
        return dx, ddelta, drate, db, dc, dskip, dgate, dbias, dstate, None, None


def _scan_inputs(x, delta, rate, b, c, skip, gate, delta_bias, lead):
    """Checks of what a scan (lead 2: steps, rows) and a step (1) share."""
    _element("x", x)
    _unit("x", x, lead + 1)
    for name, t in (("delta", delta), ("gate", gate)):
        if t is not None:
            _same(name, t, x, "x")
            _unit(name, t, lead + 1)
    D = x.shape[-1]
    if rate.dim() != 2 or not 1 <= rate.shape[1] <= 64:
        raise ValueError(f"rate must be [D, S] with S of 1 to 64, got {tuple(rate.shape)}")
    _exact("rate", rate, _f32, (D, rate.shape[1]))
    S = rate.shape[1]
    for name, t in (("b", b), ("c", c)):
        if t.dtype != x.dtype:
            raise ValueError(f"{name} must be {x.dtype}, got {t.dtype}")
        if t.dim() not in (lead + 1, lead + 2) or t.shape[:lead] != x.shape[:lead] or t.shape[-1] != S:
            raise ValueError(f"{name} must be {list(x.shape[:lead]) + [S]} or {list(x.shape[:lead]) + ['G', S]}, "
                             f"got {tuple(t.shape)}")
        _unit(name, t, t.dim())
    if b.shape != c.shape:
        raise ValueError(f"b and c must have one shape, got {tuple(b.shape)} and {tuple(c.shape)}")
    _sizes(*x.shape, *b.shape)
    if b.dim() == lead + 2 and (b.shape[lead] < 1 or D % b.shape[lead]):
        raise ValueError(f"the groups of b and c must divide the width: {b.shape[lead]} of {D}")
    _exact("skip", skip, _f32, (D,))
    _exact("delta_bias", delta_bias, _f32, (D,))


def selective_scan(x, delta, rate, b, c, skip=None, gate=None, delta_bias=None, state=None, dones=None,
                   softplus: bool = True):
    """Selective state space scan over a rollout (include/block.h): returns
    (y, new_state).  x, delta and gate (optional): [L, N, D] of one dtype
    (float32, bfloat16, float16), the last dimension contiguous, the others
    with any strides; rate: [D, S] float32, S of 1 to 64, not positive for
    decays; b, c: [L, N, S] or [L, N, G, S] of x's dtype, group g serving
    the channels from g D / G; skip, delta_bias: [D] float32; state:
    [N, D, S] float32 or None (zero); dones: [L, N] uint8 or bool, a
    collection's, or None.  The step size is softplus(delta + delta_bias), or
    delta + delta_bias itself.  y has x's dtype, new_state is float32 and
    starts the next rollout.  Gradients flow to every input but dones; a call
    that records them keeps S / 2 bytes of states for each element of x."""
    if _forward_ad._current_level >= 0:
        _no_tangent("selective_scan", x, delta, rate, b, c, skip, gate, delta_bias, state)
    _scan_inputs(x, delta, rate, b, c, skip, gate, delta_bias, 2)
    L, N, D = x.shape
    _exact("state", state, _f32, (N, D, rate.shape[1]))
    dones = _flags("dones", dones, (L, N))
    args = (x, delta, rate, b, c, skip, gate, delta_bias, state, dones, int(bool(softplus)))
    if not _wants_grad(*args[:9]):
        return _scan_forward(*args)
    return _SelectiveScan.apply(*args)


def selective_scan_step(x, delta, rate, b, c, state, skip=None, gate=None, delta_bias=None, resets=None,
                        softplus: bool = True, out_state=None):
    """One step for acting: returns (y, new_state).  As selective_scan without
    the steps' dimension: x, delta, gate: [N, D]; b, c: [N, S] or [N, G, S];
    state: [N, D, S] float32; resets: [N] uint8 or bool, rows whose episode
    ended before this step (their state counts as zero), or None.  out_state
    may be `state` itself, to update it in place.  It records no gradient."""
    if _forward_ad._current_level >= 0:
        _no_tangent("selective_scan_step", x, delta, rate, b, c, skip, gate, delta_bias, state, out_state)
    _no_grad("selective_scan_step", x, delta, rate, b, c, skip, gate, delta_bias, state, out_state)
    _scan_inputs(x, delta, rate, b, c, skip, gate, delta_bias, 1)
    N, D = x.shape
    shape = (N, D, rate.shape[1])
    _exact("state", state, _f32, shape)
    _exact("out_state", out_state, _f32, shape)
    if out_state is not None:
        _apart_or_same("out_state", out_state, state)
    resets = _flags("resets", resets, (N,))
    stream = _here("selective_scan_step", x, delta, rate, b, c, state, skip, gate, delta_bias, resets, out_state)
    y = x.new_empty((N, D))
    new = torch.empty_like(state) if out_state is None else out_state
    b_row, b_group = _strides(b, 1)
    c_row, c_group = _strides(c, 1)
    a = _SCAN(1, N, D, shape[2], b.shape[1] if b.dim() == 3 else 1, _DTYPES[x.dtype], bool(softplus),
              0, x.stride(0), 0, delta.stride(0), 0, gate.stride(0) if gate is not None else 0,
              0, b_row, b_group, 0, c_row, c_group, 0, D, x.data_ptr(), delta.data_ptr(), _at(gate), b.data_ptr(),
              c.data_ptr(), rate.data_ptr(), _at(skip), _at(delta_bias), state.data_ptr(), _at(resets), y.data_ptr(),
              new.data_ptr(), 0, 0, 0)
    _call(_entry("scan_step"), a, stream)
    if out_state is not None:
        _written(out_state)
    return y, new


# ------------------------------------------------------------- norm, dropout
def _seed(name, seed, offset):
    """(value, tensor, offset) of a seed: a number, or one int64 on the device."""
    if not 0 <= int(offset) < 1 << 32:
        raise ValueError(f"offset must be 0 to 2^32 - 1, got {offset}")
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1:
            raise ValueError(f"{name}: a seed on the device is one int64, got {seed.dtype} {tuple(seed.shape)}")
        return 0, seed, int(offset)
    return int(seed) & (1 << 64) - 1, None, int(offset)


def _probability(name, p):
    """p to the multiple of 2^-16 that the kernels use (exact in their fp32)."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"{name} must be 0 to 1, got {p}")
    return math.floor(p * 65536 + 0.5) / 65536


def _row(t):
    """Elements between rows of a contiguous tensor or of [R, D] rows."""
    return t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else t.shape[-1]


def _norm_args(residual, branch, weight, branch_weight, gate, seed_at, options):
    act, residual_scale, branch_scale, branch_norm, eps, drop, seed, offset = options
    D = residual.shape[-1]
    gate_row = 0 if gate is None or (gate.dim() == 1 and gate.dtype == _f32) else _row(gate)
    return _NORM(residual.numel() // D, D, _DTYPES[residual.dtype], branch_norm, act, residual_scale, branch_scale,
                 eps, drop, seed, _at(seed_at), offset, 0, residual.data_ptr(), _row(residual), _at(branch),
                 0 if branch is None else _row(branch), _at(gate), gate_row, _at(weight), _at(branch_weight))


def _norm_forward(residual, branch, weight, branch_weight, gate, seed_at, options, stats=None):
    where = _here("residual_norm", residual, branch, weight, branch_weight, gate, seed_at)
    stream, normed = residual.new_empty(residual.shape), residual.new_empty(residual.shape)
    D = residual.shape[-1]
    a = _norm_args(residual, branch, weight, branch_weight, gate, seed_at, options)
    _call(_entry("norm_forward"), a, stream.data_ptr(), D, normed.data_ptr(), D, _ptr(stats), where)
    return stream, normed


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, branch, weight, branch_weight, gate, seed_at, options):
        rows = residual.numel() // residual.shape[-1]
        stats = torch.empty((rows, 2), dtype=_f32, device=residual.device)
        out = _norm_forward(residual, branch, weight, branch_weight, gate, seed_at, options, stats)
        ctx.save_for_backward(residual, branch, weight, branch_weight, gate, seed_at, stats)
        ctx.options = options
        ctx.set_materialize_grads(False)
        return out

    @_first_order
    def backward(ctx, dstream, dnormed):
        residual, branch, weight, branch_weight, gate, seed_at, stats = ctx.saved_tensors
        if dstream is None and dnormed is None:
            return (None,) * 7
        lib, where = _lib(), _there(residual)
        dstream, dnormed = (None if t is None else t.contiguous() for t in (dstream, dnormed))
        f = _norm_args(residual, branch, weight, branch_weight, gate, seed_at, ctx.options)
        D, needs = residual.shape[-1], ctx.needs_input_grad

        def like(t, i):
            return t.new_empty(t.shape) if t is not None and needs[i] else None

        dresidual, dbranch, dweight, dbranch_weight, dgate = (
            like(t, i) for i, t in enumerate((residual, branch, weight, branch_weight, gate)))
        size = lib.norm_workspace(stats.shape[0], D, _DTYPES[residual.dtype])
        ws = _workspace(residual, size)
        g = f + _NORM_GRAD(stats.data_ptr(), _at(dstream), D, _at(dnormed), D, _at(dresidual), _at(dbranch),
                           _at(dgate), _at(dweight), _at(dbranch_weight), _at(ws), size)
        _call(_entry("norm_backward"), g, where)
        return dresidual, dbranch, dweight, dbranch_weight, dgate, None, None


def _norm_rows(name, t):
    if not t.is_contiguous():
        _unit(name, t, 2)
        if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError(f"{name}'s rows must not overlap")


def residual_norm(residual, branch=None, weight=None, *, branch_weight=None, gate=None, activation: str = "none",
                  residual_scale: float = 1.0, branch_scale: float = 1.0, branch_norm: bool = True,
                  eps: float = 1e-6, dropout: float = 0.0, seed=0, offset: int = 0):
    """Between two blocks (include/block.h): the branch (a block's output) is
    normed, gated, dropped and added to the residual, and the sum is normed
    for the next block; returns (stream, normed),

        stream = residual_scale residual + branch_scale drop(act(gate) rms(branch) branch_weight)
        normed = rms(stream) weight

    residual, branch: [..., D] float32, bfloat16 or float16, D of 1 to 8192,
    contiguous (or [R, D] with contiguous rows); without a branch the first
    block's norm.  weight, branch_weight: [D] float32 or None (1).
    branch_norm=False takes the branch as it is.  gate: like the branch, or
    [D] float32 for all rows; activation: "none", "sigmoid" or "silu" of the
    gate (without a gate it has no effect).  dropout, seed and offset are
    `dropout`'s on the stream's shape: two calls of one seed and offset drop the
    same places.
    Gradients flow to residual, branch, weights and gate."""
    act = _activation(activation, ("none", "sigmoid", "silu"))
    if _forward_ad._current_level >= 0:
        _no_tangent("residual_norm", residual, branch, weight, branch_weight, gate)
    _element("residual", residual)
    if residual.dim() < 1 or not 1 <= residual.shape[-1] <= 8192:
        raise ValueError(f"residual must be [..., D] with D of 1 to 8192, got {tuple(residual.shape)}")
    D = residual.shape[-1]
    _norm_rows("residual", residual)
    drop = _probability("dropout", dropout)
    seed, seed_at, offset = _seed("residual_norm", seed, offset)
    if branch is None:
        if gate is not None or branch_weight is not None or drop > 0.0:
            raise ValueError("a gate, a branch_weight or dropout needs a branch")
    else:
        _same("branch", branch, residual, "residual")
        _norm_rows("branch", branch)
    if branch_weight is not None and not branch_norm:
        raise ValueError("branch_weight needs branch_norm")
    _exact("weight", weight, _f32, (D,))
    _exact("branch_weight", branch_weight, _f32, (D,))
    if gate is not None and not (gate.dtype == _f32 and gate.shape == (D,)):
        _same("gate", gate, residual, "residual")
        _norm_rows("gate", gate)
    elif gate is not None and not gate.is_contiguous():
        raise ValueError("gate must be contiguous")
    if not float(eps) >= 0.0:
        raise ValueError(f"eps must not be negative, got {eps}")
    options = (act, float(residual_scale), float(branch_scale), int(bool(branch_norm)), float(eps), drop, seed, offset)
    args = (residual, branch, weight, branch_weight, gate, seed_at, options)
    if not _wants_grad(*args[:5]):
        return _norm_forward(*args)
    return _ResidualNorm.apply(*args)


def _drop(x, p, seed, seed_at, offset, where):
    out = torch.empty_like(x, memory_format=torch.contiguous_format)
    _call(_lib().drop_forward, _DTYPES[x.dtype], _ptr(x), x.numel(), p, seed, _ptr(seed_at), offset, _ptr(out), where)
    return out


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, seed_at, offset):
        ctx.save_for_backward(seed_at)
        ctx.draw = p, seed, offset
        return _drop(x, p, seed, seed_at, offset, _here("dropout", x, seed_at))

    @_first_order
    def backward(ctx, dout):
        seed_at, = ctx.saved_tensors
        p, seed, offset = ctx.draw
        return _drop(dout.contiguous(), p, seed, seed_at, offset, _there(dout)), None, None, None, None


def dropout(x, p: float, seed, offset: int = 0):
    """Dropout from a counter (include/block.h): each element is 0 with
    probability p (to a multiple of 2^-16), else scaled by 1 / (1 - p).
    x: a contiguous float32, bfloat16 or float16 tensor of any shape.  The
    draws depend on the seed, the offset (0 to 2^32 - 1: a layer, a call)
    and an element's place alone, and no mask is stored: the gradient draws
    again.  seed: a number, or one int64 on the device, which a captured graph
    reads anew at every replay (it must not change between a call and its
    gradient)."""
    if _forward_ad._current_level >= 0:
        _no_tangent("dropout", x)
    _element("x", x)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    p = _probability("p", p)
    seed, seed_at, offset = _seed("dropout", seed, offset)
    if not _wants_grad(x):
        return _drop(x, p, seed, seed_at, offset, _here("dropout", x, seed_at))
    return _Dropout.apply(x, p, seed, seed_at, offset)

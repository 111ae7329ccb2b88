"""Python binding of the block operators' C ABI (``include/mamba_block.h``): what makes a Mamba block and its
language model complete around the scan. The short causal convolution, the block's step from one token to the
next, the norms before and after a block, and the cross entropy over the vocabulary.

As in :mod:`.layers`, every step runs in ``libmamba_scan.so``; this module checks arguments, allocates outputs
and workspaces with torch and launches on torch's current HIP stream. There is no CPU fallback. ``<name>_fn`` is
the forward call, ``<name>_bwd`` the gradients given the incoming one, ``<name>`` the differentiable form (torch
autograd over the two; reverse mode, first derivatives). ``block_step`` is for decoding and has no gradient.
Tensors that a call writes in place (states, ``out``) must not want a gradient themselves; autograd sees that they
have changed, so that a backward pass that still needs the old values is refused.
Every call can be captured into a HIP graph, forward and backward together too; as with any torch operator, a
backward pass is captured only while no eager graph of the same leaves is alive.

Activations are float32 or bfloat16 (the cross entropy bfloat16 only); convolution weights, norm weights,
biases, ``A``, ``D``, scan states and statistics are taken in float32. Arithmetic is fp32; an activation's
gradient has the activation's dtype, a parameter's the parameter's.
"""

from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from .layers import (_dtype, _f32, _grad_on, _inner, _launch, _near_rows, _need_gpu, _on_device, _ptr, _reset, _row_stride, _rows,
                     _same, _workspace)
from .scan import load_library, refuse_graph

_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_P = ctypes.c_void_p
_F = ctypes.c_float
_I = ctypes.c_int


def _fields(pointers, sizes=(), flags=(), workspace=False):
    return [(n, _P) for n in pointers.split()] + [(n, _I64) for n in sizes] + [(n, _I32) for n in flags] + (
        [("workspace", _P), ("workspace_bytes", _I64)] if workspace else [])


def _shape(*names):
    return [(n, _I64) for n in names]


class ConvShape(ctypes.Structure):
    _fields_ = _shape("batch", "len", "dim", "width")


class ConvPtrs(ctypes.Structure):
    _fields_ = _fields("x weight bias initial_state reset y last_state", ("x_batch", "x_row", "y_batch", "y_row"), ("x_steps", "y_steps"))


class ConvBwdPtrs(ctypes.Structure):
    _fields_ = _fields("x weight bias initial_state reset dy dlast_state dx dweight dbias dinitial_state",
                       ("x_batch", "x_row", "dy_batch", "dy_row", "dx_batch", "dx_row"), ("x_steps", "dy_steps"), True)


class StepShape(ctypes.Structure):
    _fields_ = _shape("batch", "dim", "dstate", "dt_rank", "width")


class StepPtrs(ctypes.Structure):
    _fields_ = _fields("x z conv_state ssm_state conv_w conv_b w_x w_dt dt_bias A D conv_state_out ssm_state_out y",
                       ("x_stride", "z_stride"), workspace=True)


class RmsShape(ctypes.Structure):
    _fields_ = _shape("rows", "dim")


class RmsPtrs(ctypes.Structure):
    _fields_ = _fields("x residual weight y sum stats", ("x_stride", "residual_stride", "y_stride", "sum_stride"))


class RmsBwdPtrs(ctypes.Structure):
    _fields_ = _fields("t weight stats dy dsum dx dresidual dweight",
                       ("t_stride", "dy_stride", "dsum_stride", "dx_stride", "dresidual_stride"), workspace=True)


class GatedRmsShape(ctypes.Structure):
    _fields_ = _shape("rows", "dim", "groups")


class GatedRmsPtrs(ctypes.Structure):
    _fields_ = _fields("x z weight y stats", ("x_stride", "z_stride", "y_stride"))


class GatedRmsBwdPtrs(ctypes.Structure):
    _fields_ = _fields("x z weight stats dy dx dz dweight", ("x_stride", "z_stride", "dy_stride", "dx_stride", "dz_stride"),
                       workspace=True)


class XentShape(ctypes.Structure):
    _fields_ = _shape("rows", "dim", "vocab")


class XentPtrs(ctypes.Structure):
    _fields_ = _fields("x weight target loss lse total", ("x_stride", "weight_stride"), workspace=True)


class XentBwdPtrs(ctypes.Structure):
    _fields_ = _fields("x weight target lse dloss dlse dx dweight", ("x_stride", "weight_stride", "dloss_stride", "dlse_stride"),
                       workspace=True)


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    lib = load_library()
    ref = ctypes.POINTER
    for name, restype, argtypes in (
            ("mamba_block_abi_version", _I, []),
            ("mamba_conv_fwd", _I, [ref(ConvPtrs), ref(ConvShape), _I, _I, _P]),
            ("mamba_conv_bwd", _I, [ref(ConvBwdPtrs), ref(ConvShape), _I, _I, _P]),
            ("mamba_conv_bwd_workspace_bytes", _I64, [ref(ConvShape), _I, _I]),
            ("mamba_block_step", _I, [ref(StepPtrs), ref(StepShape), _I, _P]),
            ("mamba_block_step_workspace_bytes", _I64, [ref(StepShape)]),
            ("mamba_rms_norm_fwd", _I, [ref(RmsPtrs), ref(RmsShape), _F, _F, _I, _P]),
            ("mamba_rms_norm_bwd", _I, [ref(RmsBwdPtrs), ref(RmsShape), _F, _I, _P]),
            ("mamba_rms_norm_bwd_workspace_bytes", _I64, [ref(RmsShape)]),
            ("mamba_gated_rms_norm_fwd", _I, [ref(GatedRmsPtrs), ref(GatedRmsShape), _I, _F, _I, _P]),
            ("mamba_gated_rms_norm_bwd", _I, [ref(GatedRmsBwdPtrs), ref(GatedRmsShape), _I, _I, _P]),
            ("mamba_gated_rms_norm_bwd_workspace_bytes", _I64, [ref(GatedRmsShape)]),
            ("mamba_xent_fwd", _I, [ref(XentPtrs), ref(XentShape), _I, _F, _I, _P]),
            ("mamba_xent_bwd", _I, [ref(XentBwdPtrs), ref(XentShape), _I, _F, _I, _P]),
            ("mamba_xent_workspace_bytes", _I64, [ref(XentPtrs), ref(XentShape)]),
            ("mamba_xent_bwd_workspace_bytes", _I64, [ref(XentBwdPtrs), ref(XentShape)])):
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, argtypes
    _lib = lib
    return lib


def _is(t, shape, dtype, dev):
    return t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _param(t, name, shape, like, dev):
    """:func:`.layers._f32`, for the usual case in one test (a decode step's call checks ten tensors)."""
    return t if t is None or _is(t, shape, torch.float32, dev) else _f32(t, name, shape, like)


def _rows_as(t, x, name, shape, dev, dim):
    """A tensor of x's shape, dtype and device as evenly spaced rows: it, or a copy, and the stride between them."""
    if _is(t, shape, x.dtype, dev):
        return t, dim
    rows, _, stride = _rows(_same(t, x, name), name)
    return rows, stride


def _new_like(x, shape):
    """An uninitialised contiguous tensor of x's dtype (the shorter way of the two where x is one)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(shape)


def _taken(t, name, shape, dtype, dev):
    """A tensor of x's dtype and of the given shape, contiguous."""
    if not _is(t, shape, dtype, dev):
        if t.dtype is not dtype or t.get_device() != dev:
            raise TypeError(f"{name} must have x's dtype and device")
        if t.shape != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
        t = t.contiguous()
    return t


# ---- causal convolution ----

_CONV_ACTS = {None: 0, "silu": 1}


def _conv_layout(x, shape):
    """x of (batch, len, dim) as it lies: itself (copied where neither its channels nor its steps are side by
    side), the strides of its batches and rows, and whether its rows are steps of a channel."""
    batch, length, dim = x.stride()
    if dim == 1 or shape[2] <= 1:
        return x, batch, length, 0
    if length == 1 or shape[1] <= 1:
        return x, batch, dim, 1
    x = x.contiguous()
    return x, x.stride(0), x.stride(1), 0


def _new_steps(x, batch, length, dim):
    """An uninitialised (batch, len, dim) with its steps side by side: no view, so that it can be changed in place as
    a result of autograd."""
    return x.new_empty_strided((batch, length, dim), (dim * length, 1, length))


def _conv_args(x, weight, bias, activation, initial_state, reset, entry):
    dtype = _dtype(x, "x")
    if x.dim() != 3:
        raise ValueError(f"x must be (batch, len, dim), got {tuple(x.shape)}")
    if activation not in _CONV_ACTS:
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    _need_gpu(x, entry)
    batch, length, dim = x.shape
    if weight.dim() == 3 and weight.shape[1] == 1:
        weight = weight[:, 0]
    if weight.dim() != 2 or weight.shape[0] != dim or not 1 <= weight.shape[1] <= 4:
        raise ValueError(f"weight must be (dim, width) or (dim, 1, width) with dim = {dim} and width 1 to 4, got {tuple(weight.shape)}")
    width, dev = weight.shape[1], x.get_device()
    weight, bias = _param(weight, "weight", (dim, width), x, dev), _param(bias, "bias", (dim,), x, dev)
    state = None if initial_state is None else _taken(initial_state, "initial_state", (batch, width - 1, dim), x.dtype, dev)
    return dtype, _CONV_ACTS[activation], weight, bias, state, reset if reset is None else _reset(reset, batch, length, x), width


def causal_conv_fn(x, weight, bias=None, *, activation="silu", initial_state=None, reset=None, return_last_state=False,
                   scan_layout=False, out=None, last_state_out=None):
    """Short causal convolution of each channel and its activation::

        y_t = silu(bias + sum_k weight[:, k] x_{t - width + 1 + k})

    x: (batch, len, dim), float32 or bfloat16, with its channels or its steps side by side (a slice of a
    projection's output, or the scan's (batch, dim, len) transposed, is read in place). weight: (dim, width) or
    a Conv1d's (dim, 1, width), width 1 to 4. ``activation``: "silu" or None. ``initial_state``: (batch,
    width - 1, dim) in x's dtype, the inputs before the first, oldest first (default: zeros). ``reset``: (batch,
    len) bool or uint8; a set entry begins a sequence, which sees nothing from before it.

    Returns y (batch, len, dim) in x's dtype, its channels side by side as x's or, with ``scan_layout`` or where
    x's are not, its steps (``y.transpose(1, 2)`` is then what the scan takes as u); with ``return_last_state``
    also the state to go on from. ``out``: y's tensor, of that layout; ``last_state_out``: the state's, written
    whether it is returned or not, which may be ``initial_state`` itself (a decoder's state updated in place)."""
    lib = _load()
    dtype, act, weight, bias, state, reset, width = _conv_args(x, weight, bias, activation, initial_state, reset, "causal_conv_fn")
    whole = batch, length, dim = x.shape
    x, xb, xr, steps = _conv_layout(x, whole)
    y_steps = 1 if steps or scan_layout else 0
    if out is None:
        y = _new_steps(x, batch, length, dim) if y_steps else _new_like(x, whole)
    else:
        y = out
        if y.shape != whole or y.dtype is not x.dtype or y.device != x.device:
            raise ValueError("out must have x's shape, dtype and device")
        if y.stride(1 if y_steps else 2) != 1 and y.shape[1 if y_steps else 2] > 1:
            raise ValueError(f"out must have its {'steps' if y_steps else 'channels'} side by side, as y has")
        refuse_graph("out", out)
    last = last_state_out
    if last is None:
        if return_last_state:
            last = x.new_empty((batch, width - 1, dim)) if state is None else torch.empty_like(state)
    elif not _is(last, (batch, width - 1, dim), x.dtype, x.get_device()):
        raise ValueError("last_state_out must be a contiguous (batch, width - 1, dim) tensor of x's dtype and device")
    else:
        refuse_graph("last_state_out", last)
    ys = y.stride()
    ptrs = ConvPtrs(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(reset), y.data_ptr(), _ptr(last),
                    xb, xr, ys[0], ys[2 if y_steps else 1], steps, y_steps)
    _launch("mamba_conv_fwd", x, lib.mamba_conv_fwd, ptrs, ConvShape(batch, length, dim, width), act, dtype)
    if out is not None:
        increment_version(out)
    if last_state_out is not None:
        increment_version(last)
    return (y, last) if return_last_state else y


@functools.lru_cache(maxsize=64)
def _conv_bwd_bytes(batch, length, dim, width, dtype, steps, dev):
    """The gradient's workspace: by the sizes and, as workgroups are counted in compute units, the device."""
    with torch.cuda.device(dev):
        return _load().mamba_conv_bwd_workspace_bytes(ConvShape(batch, length, dim, width), dtype, steps)


def causal_conv_bwd(x, weight, bias, dy, *, activation="silu", initial_state=None, reset=None, dlast_state=None,
                    want_dinitial=None):
    """Gradients of :func:`causal_conv_fn` for incoming ``dy`` (x's shape and dtype, either layout) and,
    optionally, ``dlast_state`` (batch, width - 1, dim). Returns a dict: x in x's dtype and layout, weight
    (dim, width) in fp32, bias (fp32) where there is one, and initial_state in x's dtype when ``want_dinitial``
    (default: when one is given)."""
    lib = _load()
    dtype, act, weight, bias, state, reset, width = _conv_args(x, weight, bias, activation, initial_state, reset, "causal_conv_bwd")
    batch, length, dim = x.shape
    _same(dy, x, "dy")
    whole, dev = x.shape, x.get_device()
    x, xb, xr, steps = _conv_layout(x, whole)
    dy, gb, gr, g_steps = _conv_layout(dy, whole)
    if steps and not g_steps:
        dy = dy.transpose(1, 2).contiguous().transpose(1, 2)
        gb, gr, g_steps = dy.stride(0), dy.stride(2), 1
    dlast = None if dlast_state is None else _taken(dlast_state, "dlast_state", (batch, width - 1, dim), x.dtype, dev)
    if want_dinitial is None:
        want_dinitial = state is not None
    dx = _new_steps(x, batch, length, dim) if steps else x.new_empty(whole)
    out = {"x": dx, "weight": x.new_empty((dim, width), dtype=torch.float32)}
    if bias is not None:
        out["bias"] = x.new_empty((dim,), dtype=torch.float32)
    if want_dinitial:
        out["initial_state"] = x.new_empty((batch, width - 1, dim))
    shape, n = ConvShape(batch, length, dim, width), _conv_bwd_bytes(batch, length, dim, width, dtype, steps, dev)
    ws, ds = _workspace(n, "mamba_conv_bwd_workspace_bytes", x), dx.stride()
    ptrs = ConvBwdPtrs(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(reset), dy.data_ptr(), _ptr(dlast),
                       dx.data_ptr(), out["weight"].data_ptr(), _ptr(out.get("bias")), _ptr(out.get("initial_state")),
                       xb, xr, gb, gr, ds[0], ds[2 if steps else 1], steps, g_steps, _ptr(ws), n)
    _launch("mamba_conv_bwd", x, lib.mamba_conv_bwd, ptrs, shape, act, dtype)
    return out


class CausalConv(torch.autograd.Function):
    """y and the state after the last step, differentiable."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, reset, activation, scan_layout):
        y, last = causal_conv_fn(x, weight, bias, activation=activation, initial_state=initial_state, reset=reset,
                                 return_last_state=True, scan_layout=scan_layout)
        ctx.save_for_backward(x, weight, bias, initial_state, reset)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, weight, bias, state, reset = ctx.saved_tensors
        if dy is None and dlast is None:
            return (None,) * 7
        if dy is None:
            dy = torch.zeros_like(x)
        g = causal_conv_bwd(x, weight, bias, dy, activation=ctx.activation, initial_state=state, reset=reset, dlast_state=dlast)
        return (g["x"], g["weight"].reshape(weight.shape).to(weight.dtype), None if bias is None else g["bias"].to(bias.dtype),
                g.get("initial_state"), None, None, None)


def causal_conv(x, weight, bias=None, *, activation="silu", initial_state=None, reset=None, return_last_state=False,
                scan_layout=False):
    """Differentiable :func:`causal_conv_fn`."""
    if not _grad_on("causal_conv", x, weight, bias, initial_state):
        return causal_conv_fn(x, weight, bias, activation=activation, initial_state=initial_state, reset=reset,
                              return_last_state=return_last_state, scan_layout=scan_layout)
    y, last = CausalConv.apply(x, weight, bias, initial_state, reset, activation, scan_layout)
    return (y, last) if return_last_state else y


# ---- block step ----

@functools.lru_cache(maxsize=64)
def _step_size(batch, dim, dstate, rank, width):
    """The shape's structure and the bytes of workspace it needs (which depend on nothing else)."""
    shape = StepShape(batch, dim, dstate, rank, width)
    return shape, _load().mamba_block_step_workspace_bytes(shape)


def block_step(x, conv_state, ssm_state, conv_w, conv_b, w_x, w_dt, dt_bias, A, D=None, z=None, *, conv_state_out=None,
               ssm_state_out=None):
    """One token of each stream through a Mamba block's path from the convolution to the gate, what
    :func:`.scan.block_ssm` does for whole sequences (there with u, the projections and delta rounded to
    bfloat16, here kept in fp32)::

        u = silu(conv_b + sum_k conv_w[:, k] v_k)     v = conv_state's rows, then x
        dt, B, C = split(w_x u);  s = softplus(w_dt dt + dt_bias)
        h = exp(s A) h + s B u;  y = (C h + D u) silu(z)

    x, z: (batch, dim) float32 or bfloat16 (slices of one projection's output are read in place). conv_state:
    (batch, width - 1, dim) in x's dtype, the last inputs, oldest first (:func:`causal_conv_fn`'s state);
    ssm_state: (batch, dim, dstate) float32 (the scan's last_state). Both are updated in place, or left as they
    are and the new ones written to ``conv_state_out`` and ``ssm_state_out``. conv_w: (dim, width) or (dim, 1,
    width), width 2 to 4; w_x: (dt_rank + 2 dstate, dim) and w_dt: (dim, dt_rank) in x's dtype; conv_b, dt_bias, D: (dim,)
    or None; A: (dim, dstate). Returns y (batch, dim) in float32, as the scan does."""
    dtype = _dtype(x, "x")
    _need_gpu(x, "block_step")
    if x.dim() != 2 or ssm_state.dim() != 3 or w_dt.dim() != 2:
        raise ValueError("x must be (batch, dim), ssm_state (batch, dim, dstate) and w_dt (dim, dt_rank)")
    batch, dim = x.shape
    dstate, rank = ssm_state.shape[2], w_dt.shape[1]
    if conv_w.dim() == 3 and conv_w.shape[1] == 1:
        conv_w = conv_w[:, 0]
    if conv_w.dim() != 2 or conv_w.shape[0] != dim or not 2 <= conv_w.shape[1] <= 4:
        raise ValueError(f"conv_w must be (dim, width) with dim = {dim} and width 2 to 4, got {tuple(conv_w.shape)}")
    width = conv_w.shape[1]
    xt, per_dim, dev = x.dtype, (dim,), x.get_device()
    conv_shape, ssm_shape = (batch, width - 1, dim), (batch, dim, dstate)
    for name, t, shape, dt in (("conv_state", conv_state, conv_shape, xt), ("ssm_state", ssm_state, ssm_shape, torch.float32),
                               ("conv_state_out", conv_state_out, conv_shape, xt), ("ssm_state_out", ssm_state_out, ssm_shape, torch.float32)):
        if t is not None and not _is(t, shape, dt, dev):
            raise (TypeError if t.dtype is not dt else ValueError)(
                f"{name} must be a contiguous {dt} tensor of shape {shape} on x's device, got {t.dtype} {tuple(t.shape)}")
    conv_new, ssm_new = conv_state if conv_state_out is None else conv_state_out, ssm_state if ssm_state_out is None else ssm_state_out
    refuse_graph("conv_state" if conv_state_out is None else "conv_state_out", conv_new)
    refuse_graph("ssm_state" if ssm_state_out is None else "ssm_state_out", ssm_new)
    w_x, w_dt = _taken(w_x, "w_x", (rank + 2 * dstate, dim), xt, dev), _taken(w_dt, "w_dt", (dim, rank), xt, dev)
    if z is not None:
        z = _inner(_same(z, x, "z"))
    x = _inner(x)
    conv_w, conv_b = _param(conv_w, "conv_w", (dim, width), x, dev), _param(conv_b, "conv_b", per_dim, x, dev)
    dt_bias, A, D = _param(dt_bias, "dt_bias", per_dim, x, dev), _param(A, "A", (dim, dstate), x, dev), _param(D, "D", per_dim, x, dev)
    shape, n = _step_size(batch, dim, dstate, rank, width)
    y, ws = x.new_empty((batch, dim), dtype=torch.float32), _workspace(n, "mamba_block_step_workspace_bytes", x)
    ptrs = StepPtrs(x.data_ptr(), _ptr(z), conv_state.data_ptr(), ssm_state.data_ptr(), conv_w.data_ptr(), _ptr(conv_b),
                    w_x.data_ptr(), w_dt.data_ptr(), _ptr(dt_bias), A.data_ptr(), _ptr(D), conv_new.data_ptr(), ssm_new.data_ptr(),
                    y.data_ptr(), _row_stride(x), 0 if z is None else _row_stride(z), _ptr(ws), n)
    _launch("mamba_block_step", x, _load().mamba_block_step, ptrs, shape, dtype)
    increment_version((conv_new, ssm_new))
    return y


# ---- root-mean-square norms ----

def rms_norm_fn(x, weight=None, eps=1e-5, *, residual=None, scale=1.0, return_stats=False):
    """Root-mean-square norm over the last dimension, with the scaled residual added on the way::

        t = residual + scale x, rounded to x's dtype     (t = x without a residual, scale unused)
        y = t / sqrt(mean(t^2) + eps) * weight

    x, residual: (..., dim), float32 or bfloat16; weight: (dim,) or None. Returns y, or (y, t) with a residual;
    with ``return_stats`` a pair of that and the (rows,) fp32 inverse deviations that :func:`rms_norm_bwd`
    takes."""
    dtype = _dtype(x, "x")
    _need_gpu(x, "rms_norm_fn")
    shape, dev = x.shape, x.get_device()
    xr, rows, xs = _rows(x, "x")
    dim = shape[-1]
    rr, rs = (None, 0) if residual is None else _rows_as(residual, x, "residual", shape, dev, dim)
    weight = _param(weight, "weight", (dim,), x, dev)
    y = _new_like(x, shape)
    t = None if residual is None else _new_like(x, shape)
    stats = x.new_empty((rows,), dtype=torch.float32) if return_stats else None
    ptrs = RmsPtrs(xr.data_ptr(), _ptr(rr), _ptr(weight), y.data_ptr(), _ptr(t), _ptr(stats), xs, rs, dim, dim)
    _launch("mamba_rms_norm_fwd", x, _load().mamba_rms_norm_fwd, ptrs, RmsShape(rows, dim), scale, eps, dtype)
    out = y if residual is None else (y, t)
    return (out, stats) if return_stats else out


@functools.lru_cache(maxsize=64)
def _rms_bwd_bytes(rows, dim):
    return _load().mamba_rms_norm_bwd_workspace_bytes(RmsShape(rows, dim))


def rms_norm_bwd(t, weight, dy, stats, *, dresidual=None, scale=1.0, want_dweight=True):
    """Gradients of :func:`rms_norm_fn` at ``t`` (its x, or the sum it returned) with its ``stats``.
    ``dresidual``: the gradient that reaches t by the residual stream, added to the result; ``scale``: the
    forward's, with a residual. Returns a dict: residual (the gradient at t) and x (scale times that; the same
    tensor where scale is 1) in t's dtype, weight (fp32) where wanted."""
    dtype = _dtype(t, "t")
    _need_gpu(t, "rms_norm_bwd")
    whole, dev = t.shape, t.get_device()
    tr, rows, ts = _rows(t, "t")
    dim = whole[-1]
    gr, gs = _rows_as(dy, t, "dy", whole, dev, dim)
    rr, rs = (None, 0) if dresidual is None else _rows_as(dresidual, t, "dresidual", whole, dev, dim)
    weight, stats = _param(weight, "weight", (dim,), t, dev), _param(stats, "stats", (rows,), t, dev)
    dt = _new_like(t, whole)
    dx = _new_like(t, whole) if scale != 1.0 else None
    out = {"x": dt if dx is None else dx, "residual": dt}
    if want_dweight:
        out["weight"] = t.new_empty((dim,), dtype=torch.float32)
    n = _rms_bwd_bytes(rows, dim) if want_dweight else 0
    ws = _workspace(n, "mamba_rms_norm_bwd_workspace_bytes", t)
    ptrs = RmsBwdPtrs(tr.data_ptr(), _ptr(weight), stats.data_ptr(), gr.data_ptr(), _ptr(rr), _ptr(dx), dt.data_ptr(),
                      _ptr(out.get("weight")), ts, gs, rs, dim, dim, _ptr(ws), n)
    _launch("mamba_rms_norm_bwd", t, _load().mamba_rms_norm_bwd, ptrs, RmsShape(rows, dim), scale, dtype)
    return out


class RmsNorm(torch.autograd.Function):
    """y, and the residual stream t where a residual is given."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps, scale):
        out, stats = rms_norm_fn(x, weight, eps, residual=residual, scale=scale, return_stats=True)
        ctx.save_for_backward(x if residual is None else out[1], weight, stats)
        ctx.scale = None if residual is None else scale
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dt=None):
        t, weight, stats = ctx.saved_tensors
        if dy is None and dt is None:
            return (None,) * 5
        if dy is None:
            dy = torch.zeros_like(t)
        g = rms_norm_bwd(t, weight, dy, stats, dresidual=dt, scale=1.0 if ctx.scale is None else ctx.scale,
                         want_dweight=ctx.needs_input_grad[2])
        return (g["x"], None if ctx.scale is None else g["residual"], g["weight"].to(weight.dtype) if "weight" in g else None,
                None, None)


def rms_norm(x, weight=None, eps=1e-5, *, residual=None, scale=1.0):
    """Differentiable :func:`rms_norm_fn`: y, or (y, t) with a residual."""
    if not _grad_on("rms_norm", x, residual, weight):
        return rms_norm_fn(x, weight, eps, residual=residual, scale=scale)
    return RmsNorm.apply(x, residual, weight, eps, scale)


def _gated_args(x, z, weight, groups, entry):
    dtype = _dtype(x, "x")
    _need_gpu(x, entry)
    shape, dev = x.shape, x.get_device()
    xr, rows, xs = _rows(x, "x")
    dim = shape[-1]
    zr, zs = _rows_as(z, x, "z", shape, dev, dim)
    if groups < 1 or dim % groups:
        raise ValueError(f"groups must divide dim = {dim}, got {groups}")
    return dtype, xr, xs, zr, zs, _param(weight, "weight", (dim,), x, dev), rows, dim, shape, dev


def gated_rms_norm_fn(x, z, weight=None, eps=1e-5, *, groups=1, gate_first=True, return_stats=False):
    """The root-mean-square norm after a block's scan, with its gate z; each of ``groups`` stretches of the last
    dimension is normalised by itself::

        gate_first:  v = x silu(z),  y = v / sqrt(mean(v^2) + eps) * weight
        otherwise:   y = x / sqrt(mean(x^2) + eps) * weight * silu(z)

    x, z: (..., dim), float32 or bfloat16 (slices of one projection's output are read in place); weight: (dim,)
    or None. Returns y in x's dtype; with ``return_stats`` also the (rows, groups) fp32 inverse deviations that
    :func:`gated_rms_norm_bwd` takes."""
    dtype, xr, xs, zr, zs, weight, rows, dim, shape, _ = _gated_args(x, z, weight, groups, "gated_rms_norm_fn")
    y = _new_like(x, shape)
    stats = x.new_empty((rows, groups), dtype=torch.float32) if return_stats else None
    ptrs = GatedRmsPtrs(xr.data_ptr(), zr.data_ptr(), _ptr(weight), y.data_ptr(), _ptr(stats), xs, zs, dim)
    _launch("mamba_gated_rms_norm_fwd", x, _load().mamba_gated_rms_norm_fwd, ptrs, GatedRmsShape(rows, dim, groups), gate_first, eps,
            dtype)
    return (y, stats) if return_stats else y


@functools.lru_cache(maxsize=64)
def _gated_bwd_bytes(rows, dim, groups):
    return _load().mamba_gated_rms_norm_bwd_workspace_bytes(GatedRmsShape(rows, dim, groups))


def gated_rms_norm_bwd(x, z, weight, dy, stats, *, groups=1, gate_first=True, want_dweight=True):
    """Gradients of :func:`gated_rms_norm_fn` with its ``stats``: a dict of x and z in x's dtype, weight (fp32)
    where wanted."""
    dtype, xr, xs, zr, zs, weight, rows, dim, whole, dev = _gated_args(x, z, weight, groups, "gated_rms_norm_bwd")
    gr, gs = _rows_as(dy, x, "dy", whole, dev, dim)
    stats = _param(stats, "stats", (rows, groups), x, dev)
    out = {"x": _new_like(x, whole), "z": _new_like(x, whole)}
    if want_dweight:
        out["weight"] = x.new_empty((dim,), dtype=torch.float32)
    n = _gated_bwd_bytes(rows, dim, groups) if want_dweight else 0
    ws = _workspace(n, "mamba_gated_rms_norm_bwd_workspace_bytes", x)
    ptrs = GatedRmsBwdPtrs(xr.data_ptr(), zr.data_ptr(), _ptr(weight), stats.data_ptr(), gr.data_ptr(), out["x"].data_ptr(),
                           out["z"].data_ptr(), _ptr(out.get("weight")), xs, zs, gs, dim, dim, _ptr(ws), n)
    _launch("mamba_gated_rms_norm_bwd", x, _load().mamba_gated_rms_norm_bwd, ptrs, GatedRmsShape(rows, dim, groups), gate_first, dtype)
    return out


class GatedRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight, eps, groups, gate_first):
        y, stats = gated_rms_norm_fn(x, z, weight, eps, groups=groups, gate_first=gate_first, return_stats=True)
        ctx.save_for_backward(x, z, weight, stats)
        ctx.kw = dict(groups=groups, gate_first=gate_first)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, z, weight, stats = ctx.saved_tensors
        g = gated_rms_norm_bwd(x, z, weight, dy, stats, want_dweight=ctx.needs_input_grad[2], **ctx.kw)
        return g["x"], g["z"], g["weight"].to(weight.dtype) if "weight" in g else None, None, None, None


def gated_rms_norm(x, z, weight=None, eps=1e-5, *, groups=1, gate_first=True):
    """Differentiable :func:`gated_rms_norm_fn`."""
    if not _grad_on("gated_rms_norm", x, z, weight):
        return gated_rms_norm_fn(x, z, weight, eps, groups=groups, gate_first=gate_first)
    return GatedRmsNorm.apply(x, z, weight, eps, groups, gate_first)


# ---- cross entropy over the vocabulary ----

def _xent_args(x, weight, target, entry):
    dtype = _dtype(x, "x")
    _need_gpu(x, entry)
    shape, wshape, dev = x.shape, weight.shape, x.get_device()
    if len(shape) < 1 or len(wshape) != 2:
        raise ValueError("x must be (..., dim) and weight (vocab, dim)")
    if weight.dtype is not x.dtype or weight.get_device() != dev:
        raise TypeError("weight must have x's dtype and device")
    if wshape[1] != shape[-1]:
        raise ValueError(f"weight must be (vocab, dim) with dim = {shape[-1]}, got {tuple(wshape)}")
    ids64, lead = target.dtype is torch.int64, shape[:-1]
    if not ids64 and target.dtype is not torch.int32:
        raise TypeError(f"target must be int64 or int32, got {target.dtype}")
    if target.shape != lead or target.get_device() != dev:
        raise ValueError(f"target must be {tuple(lead)} on x's device, got {tuple(target.shape)}")
    xr, rows, xs = _rows(x, "x")
    xr, xs = _near_rows(xr, xs)
    weight = _inner(weight)
    weight, ws = _near_rows(weight, _row_stride(weight))
    return (dtype, xr, xs, weight, ws, target if target.is_contiguous() else target.contiguous(), ids64, lead, dev,
            XentShape(rows, wshape[1], wshape[0]))


def _xent_launch(name, x, f, size, ptrs, shape, *args):
    n = _on_device(x, size, ptrs, shape)
    if n != 0:
        ws = _workspace(n, name, x)
        ptrs.workspace, ptrs.workspace_bytes = ws.data_ptr(), n
    _launch(name, x, f, ptrs, shape, *args)


def _xent_fwd(x, weight, target, scale, want_lse, want_total, entry):
    lib = _load()
    dtype, xr, xs, weight, ws, target, ids64, lead, _, shape = _xent_args(x, weight, target, entry)
    loss = x.new_empty(lead, dtype=torch.float32)
    lse = x.new_empty(lead, dtype=torch.float32) if want_lse else None
    total = x.new_empty(2, dtype=torch.float32) if want_total else None
    ptrs = XentPtrs(xr.data_ptr(), weight.data_ptr(), target.data_ptr(), loss.data_ptr(), _ptr(lse), _ptr(total), xs, ws, None, 0)
    _xent_launch("mamba_xent_fwd", x, lib.mamba_xent_fwd, lib.mamba_xent_workspace_bytes, ptrs, shape, ids64, scale, dtype)
    return loss, lse, total


def linear_cross_entropy_fn(x, weight, target, *, scale=1.0, return_lse=False):
    """Softmax cross entropy of hidden states against a large output matrix, without ever storing the logits::

        l = scale x weight^T;  lse = logsumexp(l);  loss = lse - l[target]

    x: (..., dim) and weight: (vocab, dim), bfloat16; target: x.shape[:-1], int64 or int32; one outside [0,
    vocab) (such as -100) gives a loss of 0. Returns the fp32 losses of target's shape, and with ``return_lse``
    the lse that :func:`linear_cross_entropy_bwd` takes."""
    loss, lse, _ = _xent_fwd(x, weight, target, scale, return_lse, False, "linear_cross_entropy_fn")
    return (loss, lse) if return_lse else loss


def _factor(g, name, lead, dev):
    """An incoming gradient of the rows: its tensor and the stride between rows, 0 for one value for all."""
    if g is None:
        return None, 0
    if _is(g, lead, torch.float32, dev):
        return g, 1
    if g.get_device() != dev:
        raise ValueError(f"{name} must be on x's device")
    if g.shape != lead:
        raise ValueError(f"{name} must be {tuple(lead)}, got {tuple(g.shape)}")
    g = g.float()
    if g.numel() > 1 and all(s == 0 or n == 1 for n, s in zip(g.shape, g.stride())):  # broadcast from one value
        return g, 0
    return g.contiguous(), 1


def linear_cross_entropy_bwd(x, weight, target, lse, dloss, *, dlse=None, scale=1.0, want_dx=True, want_dweight=True):
    """Gradients of :func:`linear_cross_entropy_fn` with its ``lse``, for incoming ``dloss`` and, optionally,
    ``dlse``, of target's shape (either may be None). Returns a dict of x and weight in bfloat16, where wanted.
    The logits are computed again piece by piece of the vocabulary; their gradients are rounded to bfloat16
    once, as the operands of the products, without the factor of dloss where it is the same for all rows with a
    target (a mean, a sum). A row without a target or whose incoming gradients are 0 takes no
    part, whatever x holds there."""
    lib = _load()
    dtype, xr, xs, weight, ws, target, ids64, lead, dev, shape = _xent_args(x, weight, target, "linear_cross_entropy_bwd")
    lse = _param(lse, "lse", lead, x, dev)
    (a, sa), (b, sb) = _factor(dloss, "dloss", lead, dev), _factor(dlse, "dlse", lead, dev)
    out = {}
    if want_dx:
        out["x"] = _new_like(x, x.shape)
    if want_dweight:
        out["weight"] = _new_like(weight, weight.shape)
    ptrs = XentBwdPtrs(xr.data_ptr(), weight.data_ptr(), target.data_ptr(), lse.data_ptr(), _ptr(a), _ptr(b), _ptr(out.get("x")),
                       _ptr(out.get("weight")), xs, ws, sa, sb, None, 0)
    _xent_launch("mamba_xent_bwd", x, lib.mamba_xent_bwd, lib.mamba_xent_bwd_workspace_bytes, ptrs, shape, ids64, scale, dtype)
    return out


_REDUCTIONS = ("mean", "sum", "none")


def _reduced(loss, total, reduction):
    return loss if reduction == "none" else total[0] / total[1] if reduction == "mean" else total[0]


class LinearCrossEntropy(torch.autograd.Function):
    """The rows' losses, reduced, and their lse."""

    @staticmethod
    def forward(ctx, x, weight, target, scale, reduction):
        loss, lse, total = _xent_fwd(x, weight, target, scale, True, reduction != "none", "linear_cross_entropy")
        ctx.save_for_backward(x, weight, target, lse, total)
        ctx.scale, ctx.reduction = scale, reduction
        ctx.set_materialize_grads(False)
        return _reduced(loss, total, reduction), lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, dlse):
        x, weight, target, lse, total = ctx.saved_tensors
        if dloss is None and dlse is None:
            return (None,) * 5
        if dloss is not None and ctx.reduction != "none":  # one value for all rows
            dloss = (dloss / total[1] if ctx.reduction == "mean" else dloss).expand(lse.shape)
        g = linear_cross_entropy_bwd(x, weight, target, lse, dloss, dlse=dlse, scale=ctx.scale, want_dx=ctx.needs_input_grad[0],
                                     want_dweight=ctx.needs_input_grad[1])
        return g.get("x"), g.get("weight"), None, None, None


def linear_cross_entropy(x, weight, target, *, scale=1.0, reduction="mean", return_lse=False):
    """Differentiable :func:`linear_cross_entropy_fn`. ``reduction``: "mean" over the targets inside [0, vocab)
    (NaN if there are none), "sum", or "none" (the rows' losses). ``return_lse``: the rows' lse too, whose
    gradient is taken as well."""
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {_REDUCTIONS}, got {reduction!r}")
    if _grad_on("linear_cross_entropy", x, weight):
        loss, lse = LinearCrossEntropy.apply(x, weight, target, scale, reduction)
    else:
        loss, lse, total = _xent_fwd(x, weight, target, scale, return_lse, reduction != "none", "linear_cross_entropy")
        loss = _reduced(loss, total, reduction)
    return (loss, lse) if return_lse else loss

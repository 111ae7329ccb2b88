"""Python binding of the layer operators' C ABI (``include/mamba_layers.h``): the gated linear
recurrence, layer norm, the token embedding and the gated feed-forward block, each with its gradient.

As in :mod:`.scan`, every step runs in ``libmamba_scan.so``; this module checks arguments, allocates
outputs and workspaces with torch and launches on torch's current HIP stream. There is no CPU
fallback. For each operator there is

* ``<name>_fn``: the forward call;
* ``<name>_bwd``: the gradients, given the incoming one;
* ``<name>``: the differentiable form (torch autograd over the two; reverse mode, first derivatives).

Activations are float32 or bfloat16; the recurrence's ``lam``, the norm's ``weight`` and ``bias``,
states and statistics are taken in float32. Arithmetic is fp32; an activation's gradient has the
activation's dtype, a parameter's gradient the parameter's.
"""

from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from .scan import BF16, F32, _raise, load_library, refuse_graph, refuse_tangents

_I64 = ctypes.c_int64
_P = ctypes.c_void_p
_F = ctypes.c_float
_I = ctypes.c_int

GATED_CHECKPOINT = 128


class GatedShape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("len", _I64), ("dim", _I64)]


class GatedPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "r", "i", "lam", "h0", "reset", "y", "last_state", "checkpoints",
                                  "workspace")] + [("workspace_bytes", _I64)]


def _strides(*names):
    """The {batch, len} strides of the named tensors, one field each (an array field costs 0.5 us more)."""
    return [(f"{n}_{k}", _I64) for n in names for k in ("batch", "len")]


class GatedStrides(ctypes.Structure):
    _fields_ = _strides("x", "r", "i", "y")


class GatedBwdPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "r", "i", "lam", "h0", "reset", "dy", "dlast_state", "checkpoints", "dx", "dr",
                                  "di", "dlam", "dh0", "workspace")] + [("workspace_bytes", _I64)]


class GatedBwdStrides(ctypes.Structure):
    _fields_ = _strides("x", "r", "i", "dy", "dx", "dr", "di")


class NormShape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("dim", _I64)]


class NormPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "residual", "weight", "bias", "y", "sum", "stats")] + [
        (n, _I64) for n in ("x_stride", "residual_stride", "y_stride", "sum_stride")]


class NormBwdPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("t", "weight", "stats", "dy", "dresidual", "dx", "dweight", "dbias")] + [
        (n, _I64) for n in ("t_stride", "dy_stride", "dresidual_stride", "dx_stride")] + [
        ("workspace", _P), ("workspace_bytes", _I64)]


class EmbeddingShape(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("vocab", _I64), ("dim", _I64)]


class FfnShape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("dim", _I64), ("hidden", _I64)]


class FfnPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "w_gate", "w_up", "h")] + [
        (n, _I64) for n in ("x_stride", "w_gate_stride", "w_up_stride", "h_stride")] + [
        ("workspace", _P), ("workspace_bytes", _I64)]


class FfnBwdPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "w_gate", "w_up", "dh", "dx", "dw_gate", "dw_up")] + [
        (n, _I64) for n in ("x_stride", "w_gate_stride", "w_up_stride", "dh_stride")] + [
        ("workspace", _P), ("workspace_bytes", _I64)]


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    lib = load_library()
    ref = ctypes.POINTER
    for name, restype, argtypes in (
            ("mamba_layers_abi_version", _I, []),
            ("mamba_gated_scan_fwd", _I, [ref(GatedPtrs), ref(GatedShape), ref(GatedStrides), _F, _I, _P]),
            ("mamba_gated_scan_bwd", _I, [ref(GatedBwdPtrs), ref(GatedShape), ref(GatedBwdStrides), _F, _I, _P]),
            ("mamba_gated_workspace_bytes", _I64, [ref(GatedShape), _I]),
            ("mamba_gated_bwd_workspace_bytes", _I64, [ref(GatedShape), _I, _I]),
            ("mamba_layer_norm_fwd", _I, [ref(NormPtrs), ref(NormShape), _F, _I, _P]),
            ("mamba_layer_norm_bwd", _I, [ref(NormBwdPtrs), ref(NormShape), _I, _P]),
            ("mamba_layer_norm_bwd_workspace_bytes", _I64, [ref(NormShape)]),
            ("mamba_embedding_fwd", _I, [_P, _I, _P, _P, ref(EmbeddingShape), _F, _I, _P]),
            ("mamba_embedding_bwd", _I, [_P, _I, _P, _P, _P, _I64, ref(EmbeddingShape), _F, _I, _P]),
            ("mamba_embedding_bwd_workspace_bytes", _I64, [ref(EmbeddingShape)]),
            ("mamba_gated_ffn_fwd", _I, [ref(FfnPtrs), ref(FfnShape), _I, _I, _P]),
            ("mamba_gated_ffn_bwd", _I, [ref(FfnBwdPtrs), ref(FfnShape), _I, _I, _P]),
            ("mamba_gated_ffn_workspace_bytes", _I64, [ref(FfnPtrs), ref(FfnShape)]),
            ("mamba_gated_ffn_bwd_workspace_bytes", _I64, [ref(FfnShape)])):
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, argtypes
    _lib = lib
    return lib


_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _dtype(x, name):
    try:
        return _DTYPES[x.dtype]
    except KeyError:
        raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}") from None


def _need_gpu(x, entry):
    if not x.is_cuda:
        raise ValueError(f"{entry} runs on the GPU only: inputs must be device tensors")


# The handle of a device's current stream: torch's own getter where it has one (0.1 us), else by way of
# a Stream object (2 us of the 12 that a decode step's call may take).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(x, f, *args):
    """The return code of a library entry called on x's device and its current stream."""
    dev = x.get_device()
    if _current_device() == dev:
        return f(*args, _raw_stream(dev))
    with torch.cuda.device(dev):
        return f(*args, _raw_stream(dev))


def _launch(entry, x, f, *args):
    """:func:`_call`, raising what the library refuses."""
    rc = _call(x, f, *args)
    if rc != 0:
        _raise(rc, entry)


_NEEDS_WORKSPACE = -9


def _launch_maybe_workspace(entry, x, f, size, ptrs, *args):
    """:func:`_launch` of an entry that seldom needs a workspace (``size()`` bytes): tried without one
    first, as the library refuses before it enqueues anything and the query costs a short call 0.7 us."""
    rc = _call(x, f, ptrs, *args)
    if rc == _NEEDS_WORKSPACE:
        n = size()
        ws = _workspace(n, entry, x)
        ptrs.workspace, ptrs.workspace_bytes = ws.data_ptr(), n
        rc = _call(x, f, ptrs, *args)
    if rc != 0:
        _raise(rc, entry)


def _on_device(x, f, *args):
    """A size query that depends on the device it is asked for."""
    if _current_device() == x.get_device():
        return f(*args)
    with torch.cuda.device(x.get_device()):
        return f(*args)


def _f32(x, name, shape, like):
    """A parameter or state in fp32, contiguous, of the given shape (or None)."""
    if x is None:
        return None
    if x.get_device() != like.get_device():
        raise ValueError(f"{name} must be on the device of the activations")
    if x.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(x.shape)}")
    if x.dtype is not torch.float32:
        x = x.float()
    return x if x.is_contiguous() else x.contiguous()


def _ptr(x):
    return None if x is None else x.data_ptr()


def _workspace(n, entry, like):
    if n < 0:
        _raise(int(n), entry)
    return like.new_empty(n, dtype=torch.uint8) if n else None


def _same(x, like, name):
    if x.dtype is not like.dtype or x.get_device() != like.get_device():
        raise TypeError(f"{name} must have x's dtype and device")
    if x.shape != like.shape:
        raise ValueError(f"{name} must have x's shape {tuple(like.shape)}, got {tuple(x.shape)}")
    return x


def _inner(x):
    return x if x.stride(-1) == 1 or x.shape[-1] <= 1 else x.contiguous()


# ---- gated linear recurrence ----

def gated_checkpoint_shape(batch, length, dim):
    """Shape of the states that ``gated_scan_fn(checkpoints_out=)`` saves: one every 128 steps."""
    return (batch, -(-length // GATED_CHECKPOINT), dim)


def _reset(reset, batch, length, like):
    if reset is None:
        return None
    if reset.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"reset must be bool or uint8, got {reset.dtype}")
    if reset.shape != (batch, length) or reset.get_device() != like.get_device():
        raise ValueError(f"reset must be (batch, len) = {(batch, length)} on x's device")
    return reset if reset.is_contiguous() else reset.contiguous()


def _gated_sizes(x):
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x must be (batch, len, dim), got {tuple(shape)}")
    return shape


def _gated_inputs(x, r, i, lam, h0, reset, entry):
    dtype = _dtype(x, "x")
    _need_gpu(x, entry)
    batch, length, dim = _gated_sizes(x)
    return (dtype, x, _same(r, x, "r"), _same(i, x, "i"), _f32(lam, "lam", (dim,), x),
            None if h0 is None else _f32(h0, "h0", (batch, dim), x), None if reset is None else _reset(reset, batch, length, x))


_MAX_ROW_STRIDE = 1 << 21  # elements; the kernels' offsets within a run are 32-bit


def _seq(x):
    """x, copied where its last dimension is strided or its rows lie too far apart, and its strides
    {batch, len}. (Those of a dimension of one element are arbitrary in torch and never used.)"""
    batch, length, dim = x.stride()
    if (dim != 1 and x.shape[2] > 1) or (length > _MAX_ROW_STRIDE and x.shape[1] > 1):
        x = x.contiguous()
        batch, length, _ = x.stride()
    return x, batch, length


def gated_scan_fn(x, r, i, lam, *, c=8.0, h0=None, reset=None, return_last_state=False, checkpoints_out=None, out=None,
                  last_state_out=None):
    """The gated linear recurrence, one state per channel::

        log a_t = -c softplus(lam) sigmoid(r_t)          (a_t = 0 where reset)
        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,     y = h

    x, r, i: (batch, len, dim), float32 or bfloat16, unit stride along dim (slices of one projection's
    output are read in place). lam: (dim,). h0: (batch, dim) initial state or None (zero). reset:
    (batch, len) bool or uint8; a set entry forgets the state before that step (packed sequences).
    Returns y in x's dtype and, with ``return_last_state``, the fp32 state after the last step.
    ``checkpoints_out``: contiguous fp32 tensor of ``gated_checkpoint_shape`` that receives the states
    ``gated_scan_bwd(checkpoints=)`` starts from. ``out``: y's tensor; ``last_state_out``: the final
    state's, which may be ``h0`` itself (a decoder's state updated in place). Autograd sees that these three have
    changed; they must not want a gradient themselves.
    """
    lib = _load()
    dtype, x, r, i, lam, h0, reset = _gated_inputs(x, r, i, lam, h0, reset, "gated_scan_fn")
    batch, length, dim = x.shape
    (x, *xs), (r, *rs), (i, *is_) = _seq(x), _seq(r), _seq(i)
    if out is None:
        y = x.new_empty((batch, length, dim))
    else:
        y = out
        if y.shape != x.shape or y.dtype is not x.dtype or y.device != x.device or (dim > 1 and y.stride(2) != 1):
            raise ValueError("out must have x's shape, dtype and device and unit stride along dim")
        refuse_graph("out", out)
    last = None
    if return_last_state:
        last = last_state_out
        if last is None:
            last = x.new_empty((batch, dim), dtype=torch.float32)
        elif last.shape != (batch, dim) or last.dtype is not torch.float32 or last.device != x.device or not last.is_contiguous():
            raise ValueError("last_state_out must be a contiguous float32 (batch, dim) tensor on x's device")
        else:
            refuse_graph("last_state_out", last)
    if checkpoints_out is not None:
        _check_gated_checkpoints(checkpoints_out, x)
        refuse_graph("checkpoints_out", checkpoints_out)
    shape = GatedShape(batch, length, dim)
    ys = y.stride()
    ptrs = GatedPtrs(x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), _ptr(h0), _ptr(reset), y.data_ptr(), _ptr(last),
                     _ptr(checkpoints_out), None, 0)
    st = GatedStrides(*xs, *rs, *is_, ys[0], ys[1])
    _launch_maybe_workspace("mamba_gated_scan_fwd", x, lib.mamba_gated_scan_fwd,
                            lambda: _on_device(x, lib.mamba_gated_workspace_bytes, shape, dtype), ptrs, shape, st, c, dtype)
    if out is not None:
        increment_version(out)
    if return_last_state and last_state_out is not None:
        increment_version(last)
    if checkpoints_out is not None:
        increment_version(checkpoints_out)
    return (y, last) if return_last_state else y


def _check_gated_checkpoints(ck, x):
    if (ck.dtype is not torch.float32 or ck.device != x.device or tuple(ck.shape) != gated_checkpoint_shape(*x.shape)
            or not ck.is_contiguous()):
        raise ValueError(f"checkpoints must be a contiguous float32 tensor of shape {gated_checkpoint_shape(*x.shape)} "
                         f"on x's device")


def gated_scan_bwd(x, r, i, lam, dy, *, c=8.0, h0=None, reset=None, dlast_state=None, checkpoints=None, want_dh0=None):
    """Gradients of :func:`gated_scan_fn` for incoming ``dy`` (x's shape and dtype) and, optionally,
    ``dlast_state`` (batch, dim). Returns a dict: x, r, i in x's dtype, lam in fp32, and h0 in fp32
    when ``want_dh0`` (default: when h0 is given). ``checkpoints``: the states the forward saved on the
    same inputs; without them they are recomputed first. x's, r's and i's gradients are slices of one
    (batch, len, 3 dim) tensor, the gradient of a merged projection's output."""
    lib = _load()
    dtype, x, r, i, lam, h0, reset = _gated_inputs(x, r, i, lam, h0, reset, "gated_scan_bwd")
    batch, length, dim = x.shape
    (x, *xs), (r, *rs), (i, *is_), (dy, *gs) = _seq(x), _seq(r), _seq(i), _seq(_same(dy, x, "dy"))
    dlast = _f32(dlast_state, "dlast_state", (batch, dim), x)
    if checkpoints is not None:
        _check_gated_checkpoints(checkpoints, x)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    g = x.new_empty((batch, length, 3 * dim))
    dx, dr, di = g[..., :dim], g[..., dim:2 * dim], g[..., 2 * dim:]
    out = {"x": dx, "r": dr, "i": di, "lam": x.new_empty((dim,), dtype=torch.float32)}
    if want_dh0:
        out["h0"] = x.new_empty((batch, dim), dtype=torch.float32)
    shape = GatedShape(batch, length, dim)
    n = _on_device(x, lib.mamba_gated_bwd_workspace_bytes, shape, dtype, checkpoints is not None)
    ws = _workspace(n, "mamba_gated_bwd_workspace_bytes", x)
    ptrs = GatedBwdPtrs(x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), _ptr(h0), _ptr(reset), dy.data_ptr(),
                        _ptr(dlast), _ptr(checkpoints), dx.data_ptr(), dr.data_ptr(), di.data_ptr(),
                        out["lam"].data_ptr(), _ptr(out.get("h0")), _ptr(ws), n)
    t = g.stride()[:2]
    st = GatedBwdStrides(*xs, *rs, *is_, *gs, *t, *t, *t)
    _launch("mamba_gated_scan_bwd", x, lib.mamba_gated_scan_bwd, ptrs, shape, st, c, dtype)
    return out


class GatedScan(torch.autograd.Function):
    """y and the final state of the gated recurrence, differentiable."""

    @staticmethod
    def forward(ctx, x, r, i, lam, h0, c, reset):
        ck = torch.empty(gated_checkpoint_shape(*_gated_sizes(x)), dtype=torch.float32, device=x.device)
        y, last = gated_scan_fn(x, r, i, lam, c=c, h0=h0, reset=reset, return_last_state=True, checkpoints_out=ck)
        ctx.save_for_backward(x, r, i, lam, h0, reset, ck)
        ctx.c = c
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, r, i, lam, h0, reset, ck = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        g = gated_scan_bwd(x, r, i, lam, dy, c=ctx.c, h0=h0, reset=reset, dlast_state=dlast, checkpoints=ck)
        dh0 = None if h0 is None else g["h0"].to(h0.dtype)
        return g["x"], g["r"], g["i"], g["lam"].to(lam.dtype), dh0, None, None


def _grad_on(entry, *ts):
    """Whether a gradient may be asked of what is computed from these; forward-mode tangents are refused."""
    refuse_tangents(ts, entry)
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in ts)


def gated_scan(x, r, i, lam, *, c=8.0, h0=None, reset=None, return_last_state=False):
    """Differentiable :func:`gated_scan_fn`."""
    if not _grad_on("gated_scan", x, r, i, lam, h0):
        return gated_scan_fn(x, r, i, lam, c=c, h0=h0, reset=reset, return_last_state=return_last_state)
    y, last = GatedScan.apply(x, r, i, lam, h0, c, reset)
    return (y, last) if return_last_state else y


# ---- layer norm ----

def _rows(x, name):
    """x as rows of its last dimension with unit stride, without a copy where they are evenly spaced: a
    tensor that begins with them, their number and the stride between them."""
    if x.dim() != 2:
        if x.dim() == 0:
            raise ValueError(f"{name} must have at least one dimension")
        dim = x.shape[-1]
        if x.is_contiguous():  # no view made: it costs a short call 2 us
            return x, x.numel() // dim if dim else x.shape[:-1].numel(), dim
        x = x.reshape(-1, dim) if x.numel() else x.reshape(x.shape[:-1].numel(), dim)
    x = _inner(x)
    return x, x.shape[0], _row_stride(x)


def _row_stride(x):
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _near_rows(x, stride):
    """Rows for the matrix kernels, and their stride: copied where they lie further apart than a tile's 32-bit offsets
    reach (the last step of long sequences)."""
    return (x.contiguous(), x.shape[-1]) if stride > _MAX_ROW_STRIDE else (x, stride)


def layer_norm_fn(x, weight=None, bias=None, eps=1e-5, *, residual=None, return_stats=False):
    """Layer norm over the last dimension, with the residual added on the way::

        t = x + residual, rounded to x's dtype     (t = x without one)
        y = (t - mean(t)) / sqrt(var(t) + eps) * weight + bias

    x, residual: (..., dim), float32 or bfloat16; weight, bias: (dim,) or None. Returns y, or (y, t)
    with a residual; with ``return_stats`` a pair of that and the (rows, 2) fp32 means and inverse
    deviations that :func:`layer_norm_bwd` takes."""
    lib = _load()
    dtype = _dtype(x, "x")
    _need_gpu(x, "layer_norm_fn")
    shape = x.shape
    if residual is not None:
        if residual.dtype is not x.dtype or residual.get_device() != x.get_device():
            raise TypeError("residual must have x's dtype and device")
        if residual.shape != shape:
            raise ValueError(f"residual must have x's shape {tuple(shape)}, got {tuple(residual.shape)}")
    xr, rows, xs = _rows(x, "x")
    dim = shape[-1]
    rr, _, rs = (None, 0, 0) if residual is None else _rows(residual, "residual")
    weight, bias = _f32(weight, "weight", (dim,), x), _f32(bias, "bias", (dim,), x)
    y = x.new_empty(shape)
    t = None if residual is None else x.new_empty(shape)
    stats = x.new_empty((rows, 2), dtype=torch.float32) if return_stats else None
    ptrs = NormPtrs(xr.data_ptr(), _ptr(rr), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(t), _ptr(stats),
                    xs, rs, dim, dim)
    _launch("mamba_layer_norm_fwd", x, lib.mamba_layer_norm_fwd, ptrs, NormShape(rows, dim), eps, dtype)
    out = y if residual is None else (y, t)
    return (out, stats) if return_stats else out


def layer_norm_bwd(t, weight, dy, stats, *, dresidual=None, want_dweight=True, want_dbias=True):
    """Gradients of :func:`layer_norm_fn` at ``t`` (its x, or the sum it returned) with its ``stats``.
    ``dresidual``: the gradient that reaches t by the residual stream, added to the result. Returns a
    dict: x (also the residual's gradient) in t's dtype, weight and bias (fp32) where wanted."""
    lib = _load()
    dtype = _dtype(t, "t")
    _need_gpu(t, "layer_norm_bwd")
    for name, v in (("dy", dy), ("dresidual", dresidual)):
        if v is not None:
            if v.dtype is not t.dtype or v.get_device() != t.get_device():
                raise TypeError(f"{name} must have t's dtype and device")
            if v.shape != t.shape:
                raise ValueError(f"{name} must have t's shape {tuple(t.shape)}, got {tuple(v.shape)}")
    (tr, rows, ts), (gr, _, gs) = _rows(t, "t"), _rows(dy, "dy")
    rr, _, rs = (None, 0, 0) if dresidual is None else _rows(dresidual, "dresidual")
    dim = t.shape[-1]
    weight, stats = _f32(weight, "weight", (dim,), t), _f32(stats, "stats", (rows, 2), t)
    dx = t.new_empty(t.shape)
    out = {"x": dx}
    if want_dweight:
        out["weight"] = t.new_empty((dim,), dtype=torch.float32)
    if want_dbias:
        out["bias"] = t.new_empty((dim,), dtype=torch.float32)
    shape = NormShape(rows, dim)
    n = lib.mamba_layer_norm_bwd_workspace_bytes(shape) if want_dweight or want_dbias else 0
    ws = _workspace(n, "mamba_layer_norm_bwd_workspace_bytes", t)
    ptrs = NormBwdPtrs(tr.data_ptr(), _ptr(weight), stats.data_ptr(), gr.data_ptr(), _ptr(rr), dx.data_ptr(),
                       _ptr(out.get("weight")), _ptr(out.get("bias")), ts, gs, rs, dim,
                       _ptr(ws), n)
    _launch("mamba_layer_norm_bwd", t, lib.mamba_layer_norm_bwd, ptrs, shape, dtype)
    return out


class LayerNorm(torch.autograd.Function):
    """y, and the residual stream t where a residual is given."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps):
        out, stats = layer_norm_fn(x, weight, bias, eps, residual=residual, return_stats=True)
        t = x if residual is None else out[1]
        ctx.save_for_backward(t, weight, bias, stats)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dt=None):
        t, weight, bias, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None and dt is None:
            return None, None, None, None, None
        if dy is None:
            dy = torch.zeros_like(t)
        g = layer_norm_bwd(t, weight, dy, stats, dresidual=dt, want_dweight=need[2], want_dbias=need[3])
        cast = lambda name, like: g[name].to(like.dtype) if name in g else None  # noqa: E731
        return g["x"], g["x"] if ctx.has_residual else None, cast("weight", weight), cast("bias", bias), None


def layer_norm(x, weight=None, bias=None, eps=1e-5, *, residual=None):
    """Differentiable :func:`layer_norm_fn`: y, or (y, t) with a residual."""
    if not _grad_on("layer_norm", x, residual, weight, bias):
        return layer_norm_fn(x, weight, bias, eps, residual=residual)
    return LayerNorm.apply(x, residual, weight, bias, eps)


# ---- token embedding ----

def _ids(ids, like):
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"ids must be int64 or int32, got {ids.dtype}")
    if ids.get_device() != like.get_device():
        raise ValueError("ids must be on the weight's device")
    return ids if ids.is_contiguous() else ids.contiguous()


def embedding_fn(ids, weight, scale=1.0):
    """y = scale * weight[ids] in weight's dtype, shape ids.shape + (dim,). An id outside [0, vocab)
    (such as -1 for padding) gives zeros."""
    lib = _load()
    dtype = _dtype(weight, "weight")
    _need_gpu(weight, "embedding_fn")
    if weight.dim() != 2:
        raise ValueError(f"weight must be (vocab, dim), got {tuple(weight.shape)}")
    ids = _ids(ids, weight)
    weight = weight if weight.is_contiguous() else weight.contiguous()
    vocab, dim = weight.shape
    y = weight.new_empty((*ids.shape, dim))
    _launch("mamba_embedding_fwd", weight, lib.mamba_embedding_fwd, ids.data_ptr(), ids.dtype is torch.int64, weight.data_ptr(),
            y.data_ptr(), EmbeddingShape(ids.numel(), vocab, dim), scale, dtype)
    return y


def embedding_bwd(ids, dy, vocab, scale=1.0):
    """Gradient of :func:`embedding_fn` in the weight: (vocab, dim) in dy's dtype, every row written,
    each id's rows of ``dy`` added in token order in fp32."""
    lib = _load()
    dtype = _dtype(dy, "dy")
    _need_gpu(dy, "embedding_bwd")
    ids = _ids(ids, dy)
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        raise ValueError(f"dy must be ids.shape + (dim,), got {tuple(dy.shape)} for ids {tuple(ids.shape)}")
    dy = dy if dy.is_contiguous() else dy.contiguous()
    dim = dy.shape[-1]
    dw = dy.new_empty((vocab, dim))
    shape = EmbeddingShape(ids.numel(), vocab, dim)
    n = lib.mamba_embedding_bwd_workspace_bytes(shape)
    ws = _workspace(n, "mamba_embedding_bwd_workspace_bytes", dy)
    _launch("mamba_embedding_bwd", dy, lib.mamba_embedding_bwd, ids.data_ptr(), ids.dtype is torch.int64, dy.data_ptr(),
            dw.data_ptr(), _ptr(ws), n, shape, scale, dtype)
    return dw


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = weight.shape[0], scale
        return embedding_fn(ids, weight, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return None, embedding_bwd(ctx.saved_tensors[0], dy, ctx.vocab, ctx.scale), None


def embedding(ids, weight, scale=1.0):
    """Differentiable :func:`embedding_fn`."""
    return Embedding.apply(ids, weight, scale) if _grad_on("embedding", weight) else embedding_fn(ids, weight, scale)


# ---- gated feed-forward ----

_ACTS = {"silu": 0, "gelu_tanh": 1}


def _ffn_inputs(x, w_gate, w_up, activation, entry):
    dtype = _dtype(x, "x")
    _need_gpu(x, entry)
    if activation not in _ACTS:
        raise ValueError(f"activation must be one of {sorted(_ACTS)}, got {activation!r}")
    if x.dim() < 1 or w_gate.dim() != 2:
        raise ValueError("x must be (..., dim) and w_gate (hidden, dim)")
    for name, w in (("w_gate", w_gate), ("w_up", w_up)):
        if w.dtype is not x.dtype or w.get_device() != x.get_device():
            raise TypeError(f"{name} must have x's dtype and device")
        if w.dim() != 2 or w.shape != w_gate.shape or w.shape[1] != x.shape[-1]:
            raise ValueError(f"{name} must be (hidden, dim) with dim = {x.shape[-1]}, got {tuple(w.shape)}")
    xr, rows, xs = _rows(x, "x")
    xr, xs = _near_rows(xr, xs)
    wg, wu = (_near_rows(w, _row_stride(w))[0] for w in (_inner(w_gate), _inner(w_up)))
    return dtype, _ACTS[activation], xr, rows, xs, wg, wu


def gated_ffn_fn(x, w_gate, w_up, activation="silu"):
    """h = act(x w_gate^T) * (x w_up^T): both projections, the activation ("silu", or "gelu_tanh": gelu
    in its tanh form) and the product in one kernel. x: (..., dim), w_gate, w_up: (hidden, dim), all
    bfloat16; fp32 sums; returns (..., hidden) in bfloat16."""
    lib = _load()
    dtype, act, xr, rows, xs, wg, wu = _ffn_inputs(x, w_gate, w_up, activation, "gated_ffn_fn")
    hidden, dim = wg.shape
    h = x.new_empty((*x.shape[:-1], hidden))
    shape = FfnShape(rows, dim, hidden)
    ptrs = FfnPtrs(xr.data_ptr(), wg.data_ptr(), wu.data_ptr(), h.data_ptr(), xs, _row_stride(wg), _row_stride(wu),
                   hidden, None, 0)
    _launch_maybe_workspace("mamba_gated_ffn_fwd", x, lib.mamba_gated_ffn_fwd,
                            lambda: _on_device(x, lib.mamba_gated_ffn_workspace_bytes, ptrs, shape), ptrs, shape, act, dtype)
    return h


def gated_ffn_bwd(x, w_gate, w_up, dh, activation="silu"):
    """Gradients of :func:`gated_ffn_fn` for incoming dh (h's shape, bfloat16): a dict of x, w_gate and
    w_up in bfloat16. Both projections are recomputed from x; the gradients of their outputs are rounded
    to bfloat16 once, as the operands of the products."""
    lib = _load()
    dtype, act, xr, rows, xs, wg, wu = _ffn_inputs(x, w_gate, w_up, activation, "gated_ffn_bwd")
    hidden, dim = wg.shape
    if dh.dtype is not x.dtype or dh.get_device() != x.get_device():
        raise TypeError("dh must have x's dtype and device")
    if dh.shape != (*x.shape[:-1], hidden):
        raise ValueError(f"dh must be {(*x.shape[:-1], hidden)}, got {tuple(dh.shape)}")
    gr, _, gs = _rows(dh, "dh")
    out = {"x": x.new_empty(x.shape), "w_gate": x.new_empty((hidden, dim)), "w_up": x.new_empty((hidden, dim))}
    shape = FfnShape(rows, dim, hidden)
    n = _on_device(x, lib.mamba_gated_ffn_bwd_workspace_bytes, shape)
    ws = _workspace(n, "mamba_gated_ffn_bwd_workspace_bytes", x)
    ptrs = FfnBwdPtrs(xr.data_ptr(), wg.data_ptr(), wu.data_ptr(), gr.data_ptr(), out["x"].data_ptr(), out["w_gate"].data_ptr(),
                      out["w_up"].data_ptr(), xs, _row_stride(wg), _row_stride(wu), gs, _ptr(ws), n)
    _launch("mamba_gated_ffn_bwd", x, lib.mamba_gated_ffn_bwd, ptrs, shape, act, dtype)
    return out


class GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation):
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.activation = activation
        return gated_ffn_fn(x, w_gate, w_up, activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        g = gated_ffn_bwd(*ctx.saved_tensors, dh, ctx.activation)
        return g["x"], g["w_gate"], g["w_up"], None


def gated_ffn(x, w_gate, w_up, activation="silu"):
    """Differentiable :func:`gated_ffn_fn`."""
    if not _grad_on("gated_ffn", x, w_gate, w_up):
        return gated_ffn_fn(x, w_gate, w_up, activation)
    return GatedFfn.apply(x, w_gate, w_up, activation)

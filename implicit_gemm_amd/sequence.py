"""Sequence operators: the root-mean-square norm and the layer norm, the short causal convolution over tokens, the
selective state space scan and the gated delta rule, for prompts, for training (forward and gradients) and for single
tokens.

    y, h, r = rms_norm(x, w, residual)                     # and rms_norm_e4m3 for an 8-bit product behind it
    y, h, m, r = layer_norm(x, w, b, residual)
    dx, dw, db = layer_norm_grad(dy, h, w, m, r)
    y, window = causal_conv(x, w, b, silu=True)
    y, state, saved = selective_scan(u, delta, A, B, C, skip=D, z=z, delta_bias=bias, softplus=True, save=True)
    grads = selective_scan_grad(dy, u, delta, A, B, C, saved, skip=D, z=z, delta_bias=bias, softplus=True)
    y = selective_scan_step(u, delta, A, B, C, state, ...)  # one token of each sequence
    o, state, saved = gated_delta(q, k, v, g, beta, save=True)
    grads = gated_delta_grad(do, q, k, v, g, beta, saved)
    o = gated_delta_step(q, k, v, g, beta, state)

Tokens are rows and channels the contiguous last axis (of a head, where there are heads).  Sequences of one length come
as [S, L, channels]; sequences of uneven lengths as [T, channels] with `offsets` (int32 [S + 1] on the GPU, offsets[0] =
0, not decreasing; rows from offsets[S] on are padding, whose outputs are zero).  float32, bfloat16 or float16 elements,
float32 parameters (w, A, biases) and gates (g, beta), float32 states; arithmetic and sums in float32.  Rows may be strided
(a part of a wider projection).

States live in pools: `state` [P, ...] with `slots` (int32 [S] on the GPU) naming each sequence's place; without slots
sequence s has place s.  A slot outside the pool stands for no state: it reads as zeros and is not written, as the rows
that pad a batch want.  Each call runs on the current stream or `stream`; like the convolutions, a call of a gradient
is a function of its own, and there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from collections import namedtuple

import torch

from . import BF16, F16, F32, ConvWgradError, load


class _View(ctypes.Structure):
    """seq_view_t."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_int64), ("row", ctypes.c_int64)]


class _Tokens(ctypes.Structure):
    """seq_tokens_t."""
    _fields_ = [("sequences", ctypes.c_int64), ("rows", ctypes.c_int64), ("offsets", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("pool", ctypes.c_int64)]


class NormArgs(ctypes.Structure):
    """seq_norm_args_t."""
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("group", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_row", ctypes.c_int64), ("residual", ctypes.c_void_p),
                ("residual_row", ctypes.c_int64), ("w", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("rstd", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class NormGradArgs(ctypes.Structure):
    """seq_norm_grad_args_t."""
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("dy", ctypes.c_void_p), ("dy_row", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("h_row", ctypes.c_int64), ("dh", ctypes.c_void_p),
                ("dh_row", ctypes.c_int64), ("w", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dw", ctypes.c_void_p)]


class LayerNormArgs(ctypes.Structure):
    """seq_layer_norm_args_t."""
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x", ctypes.c_void_p), ("x_row", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("residual_row", ctypes.c_int64), ("w", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("y", ctypes.c_void_p), ("h", ctypes.c_void_p), ("mean", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p)]


class LayerNormGradArgs(ctypes.Structure):
    """seq_layer_norm_grad_args_t."""
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("dy", ctypes.c_void_p), ("dy_row", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("h_row", ctypes.c_int64), ("dh", ctypes.c_void_p),
                ("dh_row", ctypes.c_int64), ("w", ctypes.c_void_p), ("mean", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("dw", ctypes.c_void_p), ("db", ctypes.c_void_p)]


class ConvArgs(ctypes.Structure):
    """seq_conv_args_t."""
    _fields_ = [("tokens", _Tokens), ("channels", ctypes.c_int64), ("width", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("silu", ctypes.c_int32), ("reserved", ctypes.c_int32), ("x", _View),
                ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("state", ctypes.c_void_p),
                ("state_stride", ctypes.c_int64), ("state_out", ctypes.c_void_p),
                ("state_out_stride", ctypes.c_int64), ("y", _View)]


class ConvGradArgs(ctypes.Structure):
    """seq_conv_grad_args_t."""
    _fields_ = [("fwd", ConvArgs), ("dy", _View), ("dstate_out", ctypes.c_void_p), ("dx", _View),
                ("dw", ctypes.c_void_p), ("dbias", ctypes.c_void_p), ("dstate", ctypes.c_void_p)]


class ScanArgs(ctypes.Structure):
    """seq_scan_args_t."""
    _fields_ = [("tokens", _Tokens), ("channels", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("states", ctypes.c_int32), ("dtype", ctypes.c_int32), ("softplus", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("longest", ctypes.c_int64), ("u", _View), ("delta", _View),
                ("z", _View), ("B", _View), ("C", _View), ("B_group", ctypes.c_int64), ("C_group", ctypes.c_int64),
                ("A", ctypes.c_void_p), ("skip", ctypes.c_void_p), ("delta_bias", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("state_stride", ctypes.c_int64), ("state_out", ctypes.c_void_p),
                ("state_out_stride", ctypes.c_int64), ("save", ctypes.c_void_p), ("y", _View)]


class ScanGradArgs(ctypes.Structure):
    """seq_scan_grad_args_t."""
    _fields_ = [("fwd", ScanArgs), ("dy", _View), ("dstate_out", ctypes.c_void_p)] + \
               [(n, ctypes.c_void_p) for n in ("du", "ddelta", "dz", "dB", "dC", "dA", "dskip", "ddelta_bias", "dstate")]


class DeltaArgs(ctypes.Structure):
    """seq_delta_args_t."""
    _fields_ = [("tokens", _Tokens), ("heads", ctypes.c_int64), ("key_heads", ctypes.c_int64),
                ("key_dim", ctypes.c_int32), ("value_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q", _View), ("k", _View), ("v", _View), ("q_head", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_head", ctypes.c_int64), ("g", _View), ("beta", _View),
                ("state", ctypes.c_void_p), ("state_stride", ctypes.c_int64), ("state_out", ctypes.c_void_p),
                ("state_out_stride", ctypes.c_int64), ("save", ctypes.c_void_p), ("o", _View)]


class DeltaGradArgs(ctypes.Structure):
    """seq_delta_grad_args_t."""
    _fields_ = [("fwd", DeltaArgs), ("dout", _View), ("dout_head", ctypes.c_int64), ("dstate_out", ctypes.c_void_p)] + \
               [(n, ctypes.c_void_p) for n in ("dq", "dk", "dv", "dg", "dbeta", "dstate")]


ScanGrads = namedtuple("ScanGrads", "du ddelta dA dB dC dskip dz ddelta_bias dstate")
ScanGrads.__doc__ = """Gradients of selective_scan; None where the input was not given."""
DeltaGrads = namedtuple("DeltaGrads", "dq dk dv dg dbeta dstate")
DeltaGrads.__doc__ = """Gradients of gated_delta; dstate None without a state."""

# A call on a few tokens takes a few microseconds on the GPU, so what the host does for it counts: arguments are packed
# by one struct.pack, checks take one comparison of each property (a second function words the error), and workspace
# sizes are remembered by the sizes that they depend on.

def _format(struct_type):
    """struct format of a ctypes Structure, nested ones flattened (native alignment, as in C)."""
    codes = {ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    return "".join(codes[t] if t in codes else _format(t) for _, t in struct_type._fields_)


_NORM, _NORM_GRAD, _LAYER, _LAYER_GRAD, _CONV, _CONV_GRAD, _SCAN, _SCAN_GRAD, _DELTA, _DELTA_GRAD = (
    struct.Struct("@" + _format(t)).pack
    for t in (NormArgs, NormGradArgs, LayerNormArgs, LayerNormGradArgs, ConvArgs, ConvGradArgs, ScanArgs, ScanGradArgs,
              DeltaArgs, DeltaGradArgs))

_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_f32 = torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


@functools.lru_cache(None)
def _lib():
    """The library with the argument types of the sequence entries."""
    lib = load()
    ptr, size = ctypes.c_void_p, ctypes.c_size_t
    for name in ("seq_rms_norm", "seq_rms_norm_e4m3", "seq_layer_norm", "seq_causal_conv", "seq_causal_conv_step",
                 "seq_selective_scan_step", "seq_gated_delta_step"):
        getattr(lib, name).argtypes = [ptr, ptr]
    for name in ("seq_rms_norm_grad", "seq_layer_norm_grad", "seq_causal_conv_grad", "seq_selective_scan",
                 "seq_selective_scan_grad", "seq_gated_delta", "seq_gated_delta_grad"):
        getattr(lib, name).argtypes = [ptr, ptr, size, ptr]
    for name in ("seq_rms_norm_grad_workspace", "seq_layer_norm_grad_workspace", "seq_causal_conv_grad_workspace",
                 "seq_selective_scan_save",
                 "seq_selective_scan_workspace", "seq_selective_scan_grad_workspace", "seq_gated_delta_save",
                 "seq_gated_delta_workspace", "seq_gated_delta_grad_workspace"):
        getattr(lib, name).argtypes = [ptr, ctypes.POINTER(size)]
    return lib


def _bytes(name, packed):
    n = ctypes.c_size_t(0)
    status = getattr(_lib(), name)(packed, ctypes.byref(n))
    if status:
        raise ConvWgradError(status, name)
    return n.value


def _here(t, stream):
    """Handle of the current stream if a call on t runs there, None if it has to change stream or device first."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a GPU")
    if stream is None and index == torch.cuda.current_device():
        return _raw_stream(index)
    return None


def _there(t, stream, call, *args):
    """The call with the stream as the current one, so that what it allocates belongs to the stream that its kernels
    run on, on the device of t."""
    with torch.cuda.device(t.get_device()):
        if stream is None:
            return call(*args)
        with torch.cuda.stream(stream):
            return call(*args)


def _refuse(t, name, shape, dtype, index):
    if not isinstance(t, torch.Tensor) or t.shape != torch.Size(shape):
        raise ValueError("%s must be a tensor of shape %s, got %s" % (name, tuple(shape), getattr(t, "shape", t)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected GPU %d" % (name, t.device, index))
    raise ValueError("the last axis of %s must be contiguous" % name)


def _like(t, name, shape, dtype, index):
    """Strides of a tensor of that shape, type and device whose last axis is contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, shape, dtype, index)
    strides = t.stride()
    if strides[-1] != 1 and t.shape[-1] > 1:
        _refuse(t, name, shape, dtype, index)
    return strides


def _dense(t, name, shape, dtype, index):
    """Pointer of a contiguous tensor of that shape, type and device; 0 for None."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, shape, dtype, index)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _code(t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("elements must be float32, bfloat16 or float16, got %s" % t.dtype)
    return code


def _empty(shape, dtype, like):
    return like.new_empty(shape, dtype=dtype)


def _same(x):
    """A dense tensor of the shape and type of x."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _sequences(x, offsets, name):
    """(sequences, rows of each or in all) of [S, L, channels], or of [T, channels] with offsets."""
    shape = x.shape
    if offsets is None:
        if len(shape) != 3:
            raise ValueError("%s must be [S, L, channels] without offsets, got shape %s" % (name, tuple(shape)))
        return shape[0], shape[1]
    if len(shape) != 2:
        raise ValueError("%s must be [T, channels] with offsets, got shape %s" % (name, tuple(shape)))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must hold S + 1 >= 2 row numbers")
    return offsets.shape[0] - 1, shape[0]


def _place(t, name, P, each, dtype, index):
    """(pointer, stride between states) of a pool of P dense states."""
    if t.shape != (P,) + each or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, (P,) + each, dtype, index)
    outer, rows, one = t.stride()
    if (rows != each[1] and each[0] > 1) or (one != 1 and each[1] > 1):
        raise ValueError("each state of %s must be contiguous" % name)
    return t.data_ptr(), outer


def _pool(state, state_out, slots, S, each, dtype, index):
    """(slots, pool, state, its stride, state_out, its stride) for the arguments, after the checks of the states."""
    given = state if state is not None else state_out
    P = S if given is None else given.shape[0] if given.dim() else 0
    if P < 1:
        raise ValueError("there must be at least one sequence and one state")
    at = (0, 0) if state is None else _place(state, "state", P, each, dtype, index)
    to = at if state_out is state else (0, 0) if state_out is None else _place(state_out, "state_out", P, each, dtype, index)
    if slots is None:
        if P != S:
            raise ValueError("%d states for %d sequences: slots must say which" % (P, S))
        return 0, P, at + to
    return _dense(slots, "slots", (S,), torch.int32, index), P, at + to


def _default_out(state_out, slots, state, S, each, dtype, like):
    """Where final states go: the pool itself with slots, else a new tensor."""
    if state_out is not None:
        return state_out
    return state if slots is not None else _empty((S,) + each, dtype, like)


# ---------------------------------------------------------------------------------------------------------- norm

def _rows(t, name):
    """(row count, row stride) of [..., channels] whose rows lie a fixed distance apart."""
    shape, strides = t.shape, t.stride()
    if not shape or shape[-1] < 1:
        raise ValueError("%s must be [..., channels]" % name)
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last axis of %s must be contiguous" % name)
    if len(shape) == 2:
        return shape[0], strides[0]
    axes = [(n, s) for n, s in zip(shape[:-1], strides[:-1]) if n != 1]
    for (_, outer), (n, inner) in zip(axes, axes[1:]):
        if outer != n * inner:
            raise ValueError("the rows of %s must lie a fixed distance apart" % name)
    return t.numel() // shape[-1], axes[-1][1] if axes else shape[-1]


def _residual(residual, x, index):
    """(pointer, row stride, h pointer, h): what the addition of a residual reads and writes."""
    if residual is None:
        return 0, 0, 0, x
    if residual.shape != x.shape or residual.dtype is not x.dtype or residual.get_device() != index:
        _refuse(residual, "residual", x.shape, x.dtype, index)
    h = _same(x)
    return residual.data_ptr(), _rows(residual, "residual")[1], h.data_ptr(), h


def rms_norm(x, w, residual=None, eps=1e-5, stream=None):
    """y = h r w with h = x + residual and r = 1 / sqrt(mean(h^2) + eps) over the last axis of x [..., C]; returns
    (y, h, r).  h is rounded to the element type before the norm reads it and is x itself without a residual; w [C] and
    r [...] are float32."""
    on = _here(x, stream)
    if on is None:
        return _there(x, stream, rms_norm, x, w, residual, eps)
    shape, index, code = x.shape, x.get_device(), _code(x)
    rows, x_row = _rows(x, "x")
    res, res_row, h_ptr, h = _residual(residual, x, index)
    y, r = _same(x), _empty(shape[:-1], _f32, x)
    status = _lib().seq_rms_norm(
        _NORM(rows, shape[-1], code, 0, eps, 0, x.data_ptr(), x_row, res, res_row, _dense(w, "w", shape[-1:], _f32, index),
              y.data_ptr(), h_ptr, r.data_ptr(), 0), on)
    if status:
        raise ConvWgradError(status, "rms_norm")
    return y, h, r


def rms_norm_e4m3(x, w, residual=None, eps=1e-5, group=0, stream=None):
    """The norm of rms_norm in 8 bits: (q, scale, h) with q float8_e4m3fn [..., C] and float32 scale [..., ceil(C /
    group)], one per `group` (32, 64, 128 or 256) channels or, for group 0, one per row: scale = max|y| / 448 (1 where
    that is zero), q = y / scale, held to 448 where the scale lies below float32's normal range."""
    on = _here(x, stream)
    if on is None:
        return _there(x, stream, rms_norm_e4m3, x, w, residual, eps, group)
    shape, index, code = x.shape, x.get_device(), _code(x)
    rows, x_row = _rows(x, "x")
    C = shape[-1]
    res, res_row, h_ptr, h = _residual(residual, x, index)
    q, scale = _empty(shape, torch.float8_e4m3fn, x), _empty(shape[:-1] + (-(-C // group) if group > 0 else 1,), _f32, x)
    status = _lib().seq_rms_norm_e4m3(
        _NORM(rows, C, code, group, eps, 0, x.data_ptr(), x_row, res, res_row, _dense(w, "w", (C,), _f32, index),
              q.data_ptr(), h_ptr, 0, scale.data_ptr()), on)
    if status:
        raise ConvWgradError(status, "rms_norm_e4m3")
    return q, scale, h


@functools.lru_cache(4096)
def _norm_grad_space(rows, C, code):
    return _bytes("seq_rms_norm_grad_workspace", _NORM_GRAD(rows, C, code, *[0] * 11))


def rms_norm_grad(dy, h, w, r, dh=None, stream=None):
    """Gradients of rms_norm, from its h and r: (dx, dw).  dx is the gradient of x and of the residual alike; dh is the
    gradient that reaches h by another way (the residual stream behind it)."""
    on = _here(h, stream)
    if on is None:
        return _there(h, stream, rms_norm_grad, dy, h, w, r, dh)
    shape, dtype, index, code = h.shape, h.dtype, h.get_device(), _code(h)
    rows, h_row = _rows(h, "h")
    C = shape[-1]
    _like(dy, "dy", shape, dtype, index)
    if dh is not None:
        _like(dh, "dh", shape, dtype, index)
    dx, dw = _same(h), _empty((C,), _f32, h)
    n = _norm_grad_space(rows, C, code)
    ws = _empty(n, torch.uint8, h)
    status = _lib().seq_rms_norm_grad(
        _NORM_GRAD(rows, C, code, 0, dy.data_ptr(), _rows(dy, "dy")[1], h.data_ptr(), h_row,
                   dh.data_ptr() if dh is not None else 0, _rows(dh, "dh")[1] if dh is not None else 0,
                   _dense(w, "w", (C,), _f32, index), _dense(r, "r", shape[:-1], _f32, index), dx.data_ptr(),
                   dw.data_ptr()), ws.data_ptr(), n, on)
    if status:
        raise ConvWgradError(status, "rms_norm_grad")
    return dx, dw


def layer_norm(x, w, b=None, residual=None, eps=1e-5, stream=None):
    """y = (h - m) r w + b with h = x + residual, m = mean(h) and r = 1 / sqrt(mean((h - m)^2) + eps) over the last axis
    of x [..., C]; returns (y, h, m, r).  h is rounded to the element type before the norm reads it and is x itself
    without a residual; w, b [C] and m, r [...] are float32."""
    on = _here(x, stream)
    if on is None:
        return _there(x, stream, layer_norm, x, w, b, residual, eps)
    shape, index, code = x.shape, x.get_device(), _code(x)
    rows, x_row = _rows(x, "x")
    res, res_row, h_ptr, h = _residual(residual, x, index)
    y, m, r = _same(x), _empty(shape[:-1], _f32, x), _empty(shape[:-1], _f32, x)
    status = _lib().seq_layer_norm(
        _LAYER(rows, shape[-1], code, eps, x.data_ptr(), x_row, res, res_row, _dense(w, "w", shape[-1:], _f32, index),
               _dense(b, "b", shape[-1:], _f32, index), y.data_ptr(), h_ptr, m.data_ptr(), r.data_ptr()), on)
    if status:
        raise ConvWgradError(status, "layer_norm")
    return y, h, m, r


@functools.lru_cache(4096)
def _layer_norm_grad_space(rows, C, code):
    return _bytes("seq_layer_norm_grad_workspace", _LAYER_GRAD(rows, C, code, *[0] * 13))


def layer_norm_grad(dy, h, w, m, r, dh=None, bias=True, stream=None):
    """Gradients of layer_norm, from its h, m and r: (dx, dw, db), db None with bias false.  dx is the gradient of x and
    of the residual alike; dh is the gradient that reaches h by another way (the residual stream behind it)."""
    on = _here(h, stream)
    if on is None:
        return _there(h, stream, layer_norm_grad, dy, h, w, m, r, dh, bias)
    shape, dtype, index, code = h.shape, h.dtype, h.get_device(), _code(h)
    rows, h_row = _rows(h, "h")
    C = shape[-1]
    _like(dy, "dy", shape, dtype, index)
    if dh is not None:
        _like(dh, "dh", shape, dtype, index)
    dx, dw = _same(h), _empty((C,), _f32, h)
    db = _empty((C,), _f32, h) if bias else None
    n = _layer_norm_grad_space(rows, C, code)
    ws = _empty(n, torch.uint8, h)
    status = _lib().seq_layer_norm_grad(
        _LAYER_GRAD(rows, C, code, 0, dy.data_ptr(), _rows(dy, "dy")[1], h.data_ptr(), h_row,
                    dh.data_ptr() if dh is not None else 0, _rows(dh, "dh")[1] if dh is not None else 0,
                    _dense(w, "w", (C,), _f32, index), _dense(m, "m", shape[:-1], _f32, index),
                    _dense(r, "r", shape[:-1], _f32, index), dx.data_ptr(), dw.data_ptr(),
                    db.data_ptr() if bias else 0), ws.data_ptr(), n, on)
    if status:
        raise ConvWgradError(status, "layer_norm_grad")
    return dx, dw, db


# --------------------------------------------------------------------------------------------------- convolution

def _taps(w, D):
    if w.dim() != 2 or w.shape[0] != D or w.shape[1] < 1:
        raise ValueError("w must be [%d, taps], got shape %s" % (D, tuple(w.shape)))
    return w.shape[1]


def _conv_args(x, xs, S, L, w, b, silu, offsets, slots, state, state_out, index):
    """(taps, the arguments of seq_conv_args_t up to y); xs: (batch, row) strides of x."""
    D = x.shape[-1]
    W = _taps(w, D)
    slot_ptr, P, states = _pool(state, state_out, slots, S, (W - 1, D), x.dtype, index)
    return W, (S, L, _dense(offsets, "offsets", (S + 1,), torch.int32, index), slot_ptr, P, D, W, _code(x), bool(silu), 0,
               x.data_ptr(), *xs, _dense(w, "w", (D, W), _f32, index), _dense(b, "b", (D,), _f32, index), *states)


def _strides(t, name, offsets, index):
    """(batch, row) strides of x itself."""
    s = _like(t, name, t.shape, t.dtype, index)
    return s[:2] if offsets is None else (0, s[0])


def causal_conv(x, w, b=None, silu=False, offsets=None, slots=None, state=None, state_out=None, stream=None):
    """Short causal convolution, one filter of 2 to 4 taps per channel: y[t, d] = b[d] + sum_k w[d, k] x[t - (W - 1) +
    k, d] (times its sigmoid with silu), for x [S, L, D], or [T, D] with offsets.  Returns (y, state_out).

    `state` [P, W - 1, D] (the element type) holds the W - 1 inputs before each sequence, oldest first; None: zeros.
    The windows after the last tokens go to state_out: a new tensor by default or, with slots, `state` itself; it may
    be `state`, and must not overlap it otherwise.  causal_conv_grad reads the windows before the sequences: for a
    gradient give a state_out of its own, or keep a copy of `state`."""
    on = _here(x, stream)
    if on is None:
        return _there(x, stream, causal_conv, x, w, b, silu, offsets, slots, state, state_out)
    index = x.get_device()
    S, L = _sequences(x, offsets, "x")
    shape = x.shape
    state_out = _default_out(state_out, slots, state, S, (_taps(w, shape[-1]) - 1, shape[-1]), x.dtype, x)
    _, args = _conv_args(x, _strides(x, "x", offsets, index), S, L, w, b, silu, offsets, slots, state, state_out, index)
    y = _same(x)
    D = shape[-1]
    status = _lib().seq_causal_conv(_CONV(*args, y.data_ptr(), L * D if offsets is None else 0, D), on)
    if status:
        raise ConvWgradError(status, "causal_conv")
    return y, state_out


def causal_conv_step(x, state, w, b=None, silu=False, slots=None, state_out=None, stream=None):
    """causal_conv for one token of each sequence: x [S, D] -> y [S, D].  The new windows go to state_out, by default
    `state` itself."""
    on = _here(x, stream)
    if on is None:
        return _there(x, stream, causal_conv_step, x, state, w, b, silu, slots, state_out)
    shape, index = x.shape, x.get_device()
    if len(shape) != 2:
        raise ValueError("x must be [S, D], got shape %s" % (tuple(shape),))
    batch = _like(x, "x", shape, x.dtype, index)[0]
    _, args = _conv_args(x, (batch, 0), shape[0], 1, w, b, silu, None, slots, state,
                         state if state_out is None else state_out, index)
    y = _same(x)
    status = _lib().seq_causal_conv_step(_CONV(*args, y.data_ptr(), shape[1], 0), on)
    if status:
        raise ConvWgradError(status, "causal_conv_step")
    return y


@functools.lru_cache(4096)
def _conv_grad_space(S, L, packed, D, W, code):
    tokens = (S, L, 16 if packed else 0, 0, S)
    fwd = (*tokens, D, W, code, 0, 0, 16, 0, 0, 16, 0, 0, 0, 0, 0, 16, 0, 0)
    return _bytes("seq_causal_conv_grad_workspace", _CONV_GRAD(*fwd, *[0] * 10))


def causal_conv_grad(dy, x, w, b=None, silu=False, offsets=None, slots=None, state=None, dstate_out=None, stream=None):
    """Gradients of causal_conv: (dx, dw, db, dstate), db None without b and dstate [S, W - 1, D] None without state.
    dstate_out [S, W - 1, D]: the gradient of the outgoing windows.

    `state` holds the windows as they were before causal_conv: where that wrote the new ones over them (with slots it
    does unless told otherwise by state_out) dw and dx would be those of other inputs.  Give it a state_out of its own,
    or a copy of `state` here."""
    on = _here(x, stream)
    if on is None:
        return _there(x, stream, causal_conv_grad, dy, x, w, b, silu, offsets, slots, state, dstate_out)
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    S, L = _sequences(x, offsets, "x")
    W, args = _conv_args(x, _strides(x, "x", offsets, index), S, L, w, b, silu, offsets, slots, state, None, index)
    D = shape[-1]
    dys = _like(dy, "dy", shape, dtype, index)
    dx, dw = _same(x), _empty((D, W), _f32, x)
    db = _empty((D,), _f32, x) if b is not None else None
    dstate = _empty((S, W - 1, D), dtype, x) if state is not None else None
    n = _conv_grad_space(S, L, offsets is not None, D, W, args[7])
    ws = _empty(n, torch.uint8, x)
    status = _lib().seq_causal_conv_grad(
        _CONV_GRAD(*args, 0, 0, 0, dy.data_ptr(), *(dys[:2] if offsets is None else (0, dys[0])),
                   _dense(dstate_out, "dstate_out", (S, W - 1, D), dtype, index), dx.data_ptr(),
                   L * D if offsets is None else 0, D, dw.data_ptr(), db.data_ptr() if b is not None else 0,
                   dstate.data_ptr() if state is not None else 0), ws.data_ptr(), n, on)
    if status:
        raise ConvWgradError(status, "causal_conv_grad")
    return dx, dw, db, dstate


# ---------------------------------------------------------------------------------------------------------- scan

def _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, slots, state, state_out, max_len, S, L, step,
               index):
    """(groups, states, the arguments of seq_scan_args_t up to save)."""
    shape, dtype = u.shape, u.dtype
    D = shape[-1]
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError("A must be [%d, states], got shape %s" % (D, tuple(A.shape)))
    N = A.shape[1]
    G = B.shape[-2] if B.dim() == len(shape) + 1 else 0
    if G < 1 or D % G:
        raise ValueError("B and C must be [..., groups, states] with groups dividing %d, got %s" % (D, tuple(B.shape)))
    wide = shape[:-1] + (G, N)
    us, ds = _like(u, "u", shape, dtype, index), _like(delta, "delta", shape, dtype, index)
    Bs, Cs = _like(B, "B", wide, dtype, index), _like(C, "C", wide, dtype, index)
    zs = _like(z, "z", shape, dtype, index) if z is not None else us
    z_ptr = z.data_ptr() if z is not None else 0
    slot_ptr, P, states = _pool(state, state_out, slots, S, (D, N), _f32, index)
    if step:
        views = (u.data_ptr(), us[0], 0, delta.data_ptr(), ds[0], 0, z_ptr, zs[0], 0, B.data_ptr(), Bs[0], 0,
                 C.data_ptr(), Cs[0], 0)
    elif offsets is None:
        views = (u.data_ptr(), us[0], us[1], delta.data_ptr(), ds[0], ds[1], z_ptr, zs[0], zs[1], B.data_ptr(), Bs[0],
                 Bs[1], C.data_ptr(), Cs[0], Cs[1])
    else:
        views = (u.data_ptr(), 0, us[0], delta.data_ptr(), 0, ds[0], z_ptr, 0, zs[0], B.data_ptr(), 0, Bs[0],
                 C.data_ptr(), 0, Cs[0])
    return G, N, (S, L, _dense(offsets, "offsets", (S + 1,), torch.int32, index), slot_ptr, P, D, G, N, _code(u),
                  bool(softplus), 0, max_len or 0, *views, Bs[-2], Cs[-2], _dense(A, "A", (D, N), _f32, index),
                  _dense(skip, "skip", (D,), _f32, index), _dense(delta_bias, "delta_bias", (D,), _f32, index), *states)


def _scan_sizes(S, L, packed, D, G, N, code, longest):
    """The arguments that space depends on."""
    return (S, L, 16 if packed else 0, 0, S, D, G, N, code, 0, 0, longest, *[0] * 15, 0, 0, *[0] * 3, 0, 0, 0, 0, 0, 0, 0, 0)


@functools.lru_cache(4096)
def _scan_space(*sizes):
    """Bytes of (saved, the forward's workspace)."""
    a = _SCAN(*_scan_sizes(*sizes))
    return _bytes("seq_selective_scan_save", a), _bytes("seq_selective_scan_workspace", a)


@functools.lru_cache(4096)
def _scan_grad_space(*sizes):
    """Bytes of (saved, the gradient's workspace); fewer sizes have a gradient than a forward."""
    return _scan_space(*sizes)[0], _bytes("seq_selective_scan_grad_workspace", _SCAN_GRAD(*_scan_sizes(*sizes), *[0] * 13))


def selective_scan(u, delta, A, B, C, skip=None, z=None, delta_bias=None, softplus=False, offsets=None, max_len=None,
                   slots=None, state=None, state_out=None, save=False, stream=None):
    """Selective state space scan over u, delta, z [S, L, D], or [T, D] with offsets, with A [D, N] (float32, 1 <= N <=
    32) and B, C [S, L, G, N] or [T, G, N], channel d belonging to group d // (D / G):

        dt = delta + delta_bias, with softplus log(1 + e^dt);  h[t] = e^(dt A) h[t - 1] + dt u B[t]
        y = (sum_n h C[t] + skip u) * (z sigmoid(z) if z is given)

    Returns (y, state_out, saved).  `state` float32 [P, D, N] is where the sequences begin (None: zeros) and state_out
    where their final states go: a new tensor by default or, with slots, `state` itself; the two may be the same.
    max_len (a Python int): no sequence is longer; with offsets, whose lengths the host does not see, it spares short
    sequences the launches that split long ones.  saved is for selective_scan_grad (None without save)."""
    on = _here(u, stream)
    if on is None:
        return _there(u, stream, selective_scan, u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, max_len,
                      slots, state, state_out, save)
    index = u.get_device()
    S, L = _sequences(u, offsets, "u")
    shape = u.shape
    state_out = _default_out(state_out, slots, state, S, tuple(A.shape), _f32, u)
    G, N, args = _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, slots, state, state_out, max_len, S,
                            L, False, index)
    D = shape[-1]
    keep, n = _scan_space(S, L, offsets is not None, D, G, N, args[8], max_len or 0)
    y = _same(u)
    saved = _empty(keep // 4, _f32, u) if save else None
    ws = _empty(n, torch.uint8, u) if n else None
    status = _lib().seq_selective_scan(
        _SCAN(*args, saved.data_ptr() if save else 0, y.data_ptr(), L * D if offsets is None else 0, D),
        ws.data_ptr() if n else 0, n, on)
    if status:
        raise ConvWgradError(status, "selective_scan")
    return y, state_out, saved


def selective_scan_step(u, delta, A, B, C, state, skip=None, z=None, delta_bias=None, softplus=False, slots=None,
                        state_out=None, stream=None):
    """selective_scan for one token of each sequence: u, delta, z [S, D], B, C [S, G, N] -> y [S, D].  The new states
    go to state_out, by default `state` itself."""
    on = _here(u, stream)
    if on is None:
        return _there(u, stream, selective_scan_step, u, delta, A, B, C, state, skip, z, delta_bias, softplus, slots,
                      state_out)
    shape = u.shape
    if len(shape) != 2:
        raise ValueError("u must be [S, D], got shape %s" % (tuple(shape),))
    _, _, args = _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, None, slots, state,
                            state if state_out is None else state_out, 1, shape[0], 1, True, u.get_device())
    y = _same(u)
    status = _lib().seq_selective_scan_step(_SCAN(*args, 0, y.data_ptr(), shape[1], 0), on)
    if status:
        raise ConvWgradError(status, "selective_scan_step")
    return y


def selective_scan_grad(dy, u, delta, A, B, C, saved, skip=None, z=None, delta_bias=None, softplus=False, offsets=None,
                        max_len=None, slots=None, state=None, dstate_out=None, stream=None):
    """Gradients of selective_scan, from dy, its inputs and its `saved`: a ScanGrads tuple.  dstate_out float32 [S, D,
    N]: the gradient of the final states; dstate is that of the first ones, in the order of the sequences."""
    on = _here(u, stream)
    if on is None:
        return _there(u, stream, selective_scan_grad, dy, u, delta, A, B, C, saved, skip, z, delta_bias, softplus, offsets,
                      max_len, slots, state, dstate_out)
    shape, dtype, index = u.shape, u.dtype, u.get_device()
    S, L = _sequences(u, offsets, "u")
    G, N, args = _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, slots, state, None, max_len, S, L,
                            False, index)
    D = shape[-1]
    keep, n = _scan_grad_space(S, L, offsets is not None, D, G, N, args[8], max_len or 0)
    dys = _like(dy, "dy", shape, dtype, index)
    saved_ptr = _dense(saved, "saved", (keep // 4,), _f32, index)
    du, ddelta = _same(u), _same(u)
    dB, dC = _empty(B.shape, dtype, u), _empty(B.shape, dtype, u)
    dA = _empty((D, N), _f32, u)
    dz = _same(u) if z is not None else None
    dskip = _empty((D,), _f32, u) if skip is not None else None
    dbias = _empty((D,), _f32, u) if delta_bias is not None else None
    dstate = _empty((S, D, N), _f32, u) if state is not None else None
    ws = _empty(n, torch.uint8, u)
    status = _lib().seq_selective_scan_grad(
        _SCAN_GRAD(*args, saved_ptr, 0, 0, 0, dy.data_ptr(), *(dys[:2] if offsets is None else (0, dys[0])),
                   _dense(dstate_out, "dstate_out", (S, D, N), _f32, index), du.data_ptr(), ddelta.data_ptr(),
                   dz.data_ptr() if z is not None else 0, dB.data_ptr(), dC.data_ptr(), dA.data_ptr(),
                   dskip.data_ptr() if skip is not None else 0, dbias.data_ptr() if delta_bias is not None else 0,
                   dstate.data_ptr() if state is not None else 0), ws.data_ptr(), n, on)
    if status:
        raise ConvWgradError(status, "selective_scan_grad")
    return ScanGrads(du, ddelta, dA, dB, dC, dskip, dz, dbias, dstate)


# --------------------------------------------------------------------------------------------------- gated delta rule

def _delta_rows(v, offsets):
    """(sequences, rows of each or in all) of [S, L, H, Dv], or of [T, H, Dv] with offsets."""
    shape = v.shape
    if offsets is None:
        if len(shape) != 4:
            raise ValueError("v must be [S, L, H, Dv] without offsets, got shape %s" % (tuple(shape),))
        return shape[0], shape[1]
    if len(shape) != 3:
        raise ValueError("v must be [T, H, Dv] with offsets, got shape %s" % (tuple(shape),))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must hold S + 1 >= 2 row numbers")
    return offsets.shape[0] - 1, shape[0]


def _delta_place(t, name, P, each, index):
    """(pointer, stride between states) of a pool of P dense states [H, Dk, Dv]."""
    if t.shape != (P,) + each or t.dtype is not _f32 or t.get_device() != index:
        _refuse(t, name, (P,) + each, _f32, index)
    outer, heads, rows, one = t.stride()
    if (one != 1 and each[2] > 1) or (rows != each[2] and each[1] > 1) or (heads != each[1] * each[2] and each[0] > 1):
        raise ValueError("each state of %s must be contiguous" % name)
    return t.data_ptr(), outer


def _delta_pool(state, state_out, slots, S, each, index):
    """_pool for states of three axes."""
    given = state if state is not None else state_out
    P = S if given is None else given.shape[0] if given.dim() else 0
    if P < 1:
        raise ValueError("there must be at least one sequence and one state")
    at = (0, 0) if state is None else _delta_place(state, "state", P, each, index)
    to = at if state_out is state else (0, 0) if state_out is None else _delta_place(state_out, "state_out", P, each, index)
    if slots is None:
        if P != S:
            raise ValueError("%d states for %d sequences: slots must say which" % (P, S))
        return 0, P, at + to
    return _dense(slots, "slots", (S,), torch.int32, index), P, at + to


def _delta_keys(q, v):
    """(key heads, Dk) of q beside v."""
    H = v.shape[-2]
    if q.dim() != v.dim() or q.shape[-2] < 1 or H % q.shape[-2]:
        raise ValueError("q and k must be [..., key heads, Dk] with key heads dividing %d, got %s" % (H, tuple(q.shape)))
    return q.shape[-2:]


def _delta_args(q, k, v, g, beta, scale, offsets, slots, state, state_out, S, L, step, index):
    """The arguments of seq_delta_args_t up to save."""
    shape, dtype = v.shape, v.dtype
    H, Dv = shape[-2:]
    Hk, Dk = _delta_keys(q, v)
    keys, flat = shape[:-2] + (Hk, Dk), shape[:-1]
    qs, ks, vs = _like(q, "q", keys, dtype, index), _like(k, "k", keys, dtype, index), _like(v, "v", shape, dtype, index)
    gs, bs = _like(g, "g", flat, _f32, index), _like(beta, "beta", flat, _f32, index)
    slot_ptr, P, states = _delta_pool(state, state_out, slots, S, (H, Dk, Dv), index)
    if step:
        q_at, k_at, v_at, g_at, b_at = ((t.data_ptr(), n[0], 0) for t, n in ((q, qs), (k, ks), (v, vs), (g, gs), (beta, bs)))
    elif offsets is None:
        q_at, k_at, v_at, g_at, b_at = ((t.data_ptr(), n[0], n[1])
                                        for t, n in ((q, qs), (k, ks), (v, vs), (g, gs), (beta, bs)))
    else:
        q_at, k_at, v_at, g_at, b_at = ((t.data_ptr(), 0, n[0]) for t, n in ((q, qs), (k, ks), (v, vs), (g, gs), (beta, bs)))
    return (S, L, _dense(offsets, "offsets", (S + 1,), torch.int32, index), slot_ptr, P, H, Hk, Dk, Dv, _code(v),
            Dk ** -0.5 if scale is None else scale, *q_at, *k_at, *v_at, qs[-2], ks[-2], vs[-2], *g_at, *b_at, *states)


def _delta_sizes(S, L, packed, H, Hk, Dk, Dv, code):
    """The arguments that space depends on."""
    return (S, L, 16 if packed else 0, 0, S, H, Hk, Dk, Dv, code, 0.0, *[0] * 9, 0, 0, 0, *[0] * 6, 0, 0, 0, 0, 0, 0, 0, 0)


@functools.lru_cache(4096)
def _delta_space(*sizes):
    """Bytes of (saved, the forward's workspace)."""
    a = _DELTA(*_delta_sizes(*sizes))
    return _bytes("seq_gated_delta_save", a), _bytes("seq_gated_delta_workspace", a)


@functools.lru_cache(4096)
def _delta_grad_space(*sizes):
    """Bytes of (saved, the gradient's workspace)."""
    return _delta_space(*sizes)[0], _bytes("seq_gated_delta_grad_workspace", _DELTA_GRAD(*_delta_sizes(*sizes), *[0] * 11))


def gated_delta(q, k, v, g, beta, scale=None, offsets=None, slots=None, state=None, state_out=None, save=False,
                stream=None):
    """Gated delta rule over q, k [S, L, Hk, Dk], v [S, L, H, Dv] and float32 g, beta [S, L, H], or the same without S
    with offsets; heads of v share those of q and k, head h having key head h // (H / Hk):

        S = e^g S;  S = S + beta k (v - S^T k)^T;  o = scale S^T q        (scale: Dk ** -0.5 by default)

    per token and head with a state S [Dk, Dv].  g is the logarithm of a decay (<= 0 as a rule; else results have 32 bits of
    what 64 tokens would grow to by their g alone), keys have unit length as a rule.  Dk <= 256, Dv <= 1024.  An element
    that is not finite reaches its token's output (q), its column of the head's outputs from its token on (v), all of them
    (k, beta, and g but for -inf), or its column of all outputs of the sequence (state); v, k, beta and g possibly also the
    up to 63 tokens before theirs.

    Returns (o, state_out, saved).  `state` float32 [P, H, Dk, Dv] is where the sequences begin (None: zeros) and
    state_out where their final states go: a new tensor by default or, with slots, `state` itself; the two may be the
    same, and must not overlap otherwise.  saved is for gated_delta_grad (None without save)."""
    on = _here(v, stream)
    if on is None:
        return _there(v, stream, gated_delta, q, k, v, g, beta, scale, offsets, slots, state, state_out, save)
    index = v.get_device()
    S, L = _delta_rows(v, offsets)
    shape = v.shape
    H, Dv = shape[-2:]
    Hk, Dk = _delta_keys(q, v)
    keep, n = _delta_space(S, L, offsets is not None, H, Hk, Dk, Dv, _code(v))     # refuses sizes before they are allocated
    state_out = _default_out(state_out, slots, state, S, (H, Dk, Dv), _f32, v)
    args = _delta_args(q, k, v, g, beta, scale, offsets, slots, state, state_out, S, L, False, index)
    o = _same(v)
    saved = _empty(keep // 4, _f32, v) if save else None
    ws = _empty(n, torch.uint8, v)
    status = _lib().seq_gated_delta(
        _DELTA(*args, saved.data_ptr() if save else 0, o.data_ptr(), L * H * Dv if offsets is None else 0, H * Dv),
        ws.data_ptr(), n, on)
    if status:
        raise ConvWgradError(status, "gated_delta")
    return o, state_out, saved


def gated_delta_step(q, k, v, g, beta, state, scale=None, slots=None, state_out=None, stream=None):
    """gated_delta for one token of each sequence: q, k [S, Hk, Dk], v [S, H, Dv], g, beta [S, H] -> o [S, H, Dv].  The
    new states go to state_out, by default `state` itself."""
    on = _here(v, stream)
    if on is None:
        return _there(v, stream, gated_delta_step, q, k, v, g, beta, state, scale, slots, state_out)
    shape = v.shape
    if len(shape) != 3:
        raise ValueError("v must be [S, H, Dv], got shape %s" % (tuple(shape),))
    args = _delta_args(q, k, v, g, beta, scale, None, slots, state, state if state_out is None else state_out, shape[0], 1,
                       True, v.get_device())
    o = _same(v)
    status = _lib().seq_gated_delta_step(_DELTA(*args, 0, o.data_ptr(), shape[1] * shape[2], 0), on)
    if status:
        raise ConvWgradError(status, "gated_delta_step")
    return o


def gated_delta_grad(do, q, k, v, g, beta, saved, scale=None, offsets=None, slots=None, state=None, dstate_out=None,
                     stream=None):
    """Gradients of gated_delta, from do, its inputs and its `saved`: a DeltaGrads tuple.  dstate_out float32 [S, H, Dk,
    Dv]: the gradient of the final states; dstate is that of the first ones, in the order of the sequences.  dg is a sum in
    which what a token writes itself cancels: it is good to 32 bits of those terms (|do| |o| and |dv| |v| of its chunk), so that
    a dg of zero, as of a first token without a state, comes out as their rounding."""
    on = _here(v, stream)
    if on is None:
        return _there(v, stream, gated_delta_grad, do, q, k, v, g, beta, saved, scale, offsets, slots, state, dstate_out)
    shape, dtype, index = v.shape, v.dtype, v.get_device()
    S, L = _delta_rows(v, offsets)
    H, Dv = shape[-2:]
    args = _delta_args(q, k, v, g, beta, scale, offsets, slots, state, None, S, L, False, index)
    Dk = args[7]
    keep, n = _delta_grad_space(S, L, offsets is not None, H, *args[6:10])
    dos = _like(do, "do", shape, dtype, index)
    saved_ptr = _dense(saved, "saved", (keep // 4,), _f32, index)
    dq, dk, dv = _empty(q.shape, dtype, v), _empty(q.shape, dtype, v), _same(v)
    dg, dbeta = _empty(shape[:-1], _f32, v), _empty(shape[:-1], _f32, v)
    dstate = _empty((S, H, Dk, Dv), _f32, v) if state is not None else None
    ws = _empty(n, torch.uint8, v)
    status = _lib().seq_gated_delta_grad(
        _DELTA_GRAD(*args, saved_ptr, 0, 0, 0, do.data_ptr(), *(dos[:2] if offsets is None else (0, dos[0])), dos[-2],
                    _dense(dstate_out, "dstate_out", (S, H, Dk, Dv), _f32, index), dq.data_ptr(), dk.data_ptr(),
                    dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), dstate.data_ptr() if state is not None else 0),
        ws.data_ptr(), n, on)
    if status:
        raise ConvWgradError(status, "gated_delta_grad")
    return DeltaGrads(dq, dk, dv, dg, dbeta, dstate)

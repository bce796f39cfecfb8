"""Sequence operators: the root-mean-square norm, the short causal convolution over tokens and the selective state
space scan, for prompts, for training (forward and gradients) and for single tokens.

    y, h, r = rms_norm(x, w, residual)                     # and rms_norm_e4m3 for an 8-bit product behind it
    y, window = causal_conv(x, w, b, silu=True)
    y, state, saved = selective_scan(u, delta, A, B, C, skip=D, z=z, delta_bias=bias, softplus=True, save=True)
    grads = selective_scan_grad(dy, u, delta, A, B, C, saved, skip=D, z=z, delta_bias=bias, softplus=True)
    y = selective_scan_step(u, delta, A, B, C, state, ...)  # one token of each sequence

Tokens are rows and channels the contiguous last axis.  Sequences of one length come as [S, L, channels]; sequences of
uneven lengths as [T, channels] with `offsets` (int32 [S + 1] on the GPU, offsets[0] = 0, not decreasing; rows from
offsets[S] on are padding, whose outputs are zero).  float32, bfloat16 or float16 elements, float32 parameters (w, A,
biases), float32 scan states; arithmetic and sums in float32.  Rows may be strided (a part of a wider projection).

States live in pools: `state` [P, ...] with `slots` (int32 [S] on the GPU) naming each sequence's place; without slots
sequence s has place s.  A slot outside the pool stands for no state: it reads as zeros and is not written, as the rows
that pad a batch want.  Each call runs on the current stream or `stream`; like the convolutions, a call of a gradient
is a function of its own, and there is no fallback.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import ConvWgradError, _dtype_code, load


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


ScanGrads = namedtuple("ScanGrads", "du ddelta dA dB dC dskip dz ddelta_bias dstate")
ScanGrads.__doc__ = """Gradients of selective_scan; None where the input was not given."""

_bound = None


def _lib():
    """The library with the argument types of the sequence entries."""
    global _bound
    if _bound is None:
        lib = load()
        P, ptr, size = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
        for name, args in (("seq_rms_norm", NormArgs), ("seq_rms_norm_e4m3", NormArgs), ("seq_causal_conv", ConvArgs),
                           ("seq_causal_conv_step", ConvArgs), ("seq_selective_scan_step", ScanArgs)):
            getattr(lib, name).argtypes = [P(args), ptr]
        for name, args in (("seq_rms_norm_grad", NormGradArgs), ("seq_causal_conv_grad", ConvGradArgs),
                           ("seq_selective_scan", ScanArgs), ("seq_selective_scan_grad", ScanGradArgs)):
            getattr(lib, name).argtypes = [P(args), ptr, size, ptr]
        for name, args in (("seq_rms_norm_grad_workspace", NormGradArgs),
                           ("seq_causal_conv_grad_workspace", ConvGradArgs), ("seq_selective_scan_save", ScanArgs),
                           ("seq_selective_scan_workspace", ScanArgs),
                           ("seq_selective_scan_grad_workspace", ScanGradArgs)):
            getattr(lib, name).argtypes = [P(args), P(size)]
        _bound = lib
    return _bound


def _check(status, what):
    if status:
        raise ConvWgradError(status, what)


def _bytes(name, args):
    n = ctypes.c_size_t(0)
    _check(getattr(_lib(), name)(ctypes.byref(args), ctypes.byref(n)), name)
    return n.value


class _On:
    """The stream of a call as the current one, on the device of its tensors (nothing to do where it already is):
    outputs and workspaces allocated inside belong to the stream that the kernels run on."""

    def __init__(self, t, stream):
        if not t.is_cuda:
            raise ValueError("tensors must be on a GPU")
        self.guards = []
        index = t.device.index
        if index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(index))
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
        self.stream = stream
        self.device = t.device

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return (self.stream or torch.cuda.current_stream(self.device)).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _like(t, name, shape, dtype, device):
    """A tensor of that shape, type and device whose last axis is contiguous."""
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be a tensor of shape %s, got %s" % (name, tuple(shape), getattr(t, "shape", t)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the last axis of %s must be contiguous" % name)
    return t


def _param(t, name, shape, device):
    """Pointer of a contiguous float32 parameter, 0 for None."""
    if t is None:
        return 0
    _like(t, name, shape, torch.float32, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _dense(t, name, shape, dtype, device):
    _like(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _view(t, packed):
    """seq_view_t of [S, L, ...] or, packed, [T, ...]."""
    return (t.data_ptr(), 0, t.stride(0)) if packed else (t.data_ptr(), t.stride(0), t.stride(1))


def _index(t, name, n, device):
    if t is None:
        return 0
    if t.dtype != torch.int32 or tuple(t.shape) != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape (%d,) on %s" % (name, n, device))
    return t.data_ptr()


def _sequences(x, offsets, name):
    """(packed, sequences, rows) of [S, L, channels], or of [T, channels] with offsets."""
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("%s must be [S, L, channels] without offsets, got shape %s" % (name, tuple(x.shape)))
        return False, x.shape[0], x.shape[1]
    if x.dim() != 2:
        raise ValueError("%s must be [T, channels] with offsets, got shape %s" % (name, tuple(x.shape)))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must hold S + 1 >= 2 row numbers")
    return True, offsets.shape[0] - 1, x.shape[0]


def _pool(state, state_out, slots, S, each, dtype, device):
    """(slots pointer, pool) after the checks of the states and slots of a call."""
    pools = {t.shape[0] for t in (state, state_out) if t is not None and t.dim() == 1 + len(each)}
    if len(pools) > 1:
        raise ValueError("state and state_out must hold the same number of states")
    P = pools.pop() if pools else S
    for t, name in ((state, "state"), (state_out, "state_out")):
        if t is not None:
            _like(t, name, (P,) + each, dtype, device)
            if t.shape[0] and not t[0].is_contiguous():
                raise ValueError("each state of %s must be contiguous" % name)
    if slots is None and P != S:
        raise ValueError("%d states for %d sequences: slots must say which" % (P, S))
    if P == 0:
        raise ValueError("the pool is empty")
    return _index(slots, "slots", S, device), P


def _state(t):
    return (0, 0) if t is None else (t.data_ptr(), t.stride(0))


# ---------------------------------------------------------------------------------------------------------- norm

def _rows(t, name):
    """(row count, row stride) of [..., channels] whose rows lie a fixed distance apart."""
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError("%s must be [..., channels]" % name)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the last axis of %s must be contiguous" % name)
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    if t.dim() == 1:
        return 1, t.shape[0]
    rows = t.numel() // t.shape[-1]
    axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    for (_, outer), (n, inner) in zip(axes, axes[1:]):
        if outer != n * inner:
            raise ValueError("the rows of %s must lie a fixed distance apart" % name)
    return rows, axes[-1][1] if axes else t.shape[-1]


def _norm_args(x, w, residual, eps, group):
    dtype = _dtype_code(x)
    rows, x_row = _rows(x, "x")
    C = x.shape[-1]
    res_row = 0
    if residual is not None:
        _like(residual, "residual", x.shape, x.dtype, x.device)
        res_row = _rows(residual, "residual")[1]
    return rows, NormArgs(rows, C, dtype, group, eps, 0, x.data_ptr(), x_row,
                          residual.data_ptr() if residual is not None else 0, res_row, _param(w, "w", (C,), x.device))


def rms_norm(x, w, residual=None, eps=1e-5, stream=None):
    """y = h r w with h = x + residual and r = 1 / sqrt(mean(h^2) + eps) over the last axis of x [..., C]; returns
    (y, h, r).  h is rounded to the element type before the norm reads it and is x itself without a residual; w [C] and
    r [...] are float32."""
    with _On(x, stream) as s:
        rows, a = _norm_args(x, w, residual, eps, 0)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        r = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        h = x
        if residual is not None:
            h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            a.h = h.data_ptr()
        a.y, a.rstd = y.data_ptr(), r.data_ptr()
        _check(_lib().seq_rms_norm(ctypes.byref(a), s), "rms_norm")
    return y, h, r


def rms_norm_e4m3(x, w, residual=None, eps=1e-5, group=0, stream=None):
    """The norm of rms_norm in 8 bits: (q, scale, h) with q float8_e4m3fn [..., C] and float32 scale [..., ceil(C /
    group)], one per `group` (32, 64, 128 or 256) channels or, for group 0, one per row: scale = max|y| / 448 (1 where
    that is zero), q = y / scale."""
    with _On(x, stream) as s:
        rows, a = _norm_args(x, w, residual, eps, group)
        C = x.shape[-1]
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(x.shape[:-1] + (-(-C // group) if group else 1,), dtype=torch.float32, device=x.device)
        h = x
        if residual is not None:
            h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            a.h = h.data_ptr()
        a.y, a.scale = q.data_ptr(), scale.data_ptr()
        _check(_lib().seq_rms_norm_e4m3(ctypes.byref(a), s), "rms_norm_e4m3")
    return q, scale, h


def rms_norm_grad(dy, h, w, r, dh=None, stream=None):
    """Gradients of rms_norm, from its h and r: (dx, dw).  dx is the gradient of x and of the residual alike; dh is the
    gradient that reaches h by another way (the residual stream behind it)."""
    with _On(h, stream) as s:
        dtype = _dtype_code(h)
        rows, h_row = _rows(h, "h")
        C = h.shape[-1]
        _like(dy, "dy", h.shape, h.dtype, h.device)
        if dh is not None:
            _like(dh, "dh", h.shape, h.dtype, h.device)
        if r.dtype != torch.float32 or r.shape != h.shape[:-1] or r.device != h.device or not r.is_contiguous():
            raise ValueError("r must be what rms_norm returned for h")
        a = NormGradArgs(rows, C, dtype, 0, dy.data_ptr(), _rows(dy, "dy")[1], h.data_ptr(), h_row,
                         dh.data_ptr() if dh is not None else 0, _rows(dh, "dh")[1] if dh is not None else 0,
                         _param(w, "w", (C,), h.device), r.data_ptr())
        dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
        dw = torch.empty((C,), dtype=torch.float32, device=h.device)
        a.dx, a.dw = dx.data_ptr(), dw.data_ptr()
        n = _bytes("seq_rms_norm_grad_workspace", a)
        ws = torch.empty(n, dtype=torch.uint8, device=h.device)
        _check(_lib().seq_rms_norm_grad(ctypes.byref(a), ws.data_ptr(), n, s), "rms_norm_grad")
    return dx, dw


# --------------------------------------------------------------------------------------------------- convolution

def _conv_args(x, w, b, silu, offsets, slots, state, state_out, name="x"):
    packed, S, L = _sequences(x, offsets, name)
    D = x.shape[-1]
    if w.dim() != 2 or w.shape[0] != D:
        raise ValueError("w must be [%d, taps], got shape %s" % (D, tuple(w.shape)))
    W = w.shape[1]
    _like(x, name, x.shape, x.dtype, x.device)
    slot_ptr, P = _pool(state, state_out, slots, S, (W - 1, D), x.dtype, x.device)
    tokens = (S, L, _index(offsets, "offsets", S + 1, x.device), slot_ptr, P)
    a = ConvArgs(tokens, D, W, _dtype_code(x), bool(silu), 0, _view(x, packed), _param(w, "w", (D, W), x.device),
                 _param(b, "b", (D,), x.device), *_state(state), *_state(state_out))
    return packed, S, a


def causal_conv(x, w, b=None, silu=False, offsets=None, slots=None, state=None, state_out=None, stream=None):
    """Short causal convolution, one filter of 2 to 4 taps per channel: y[t, d] = b[d] + sum_k w[d, k] x[t - (W - 1) +
    k, d] (times its sigmoid with silu), for x [S, L, D], or [T, D] with offsets.  Returns (y, state_out).

    `state` [P, W - 1, D] (the element type) holds the W - 1 inputs before each sequence, oldest first; None: zeros.
    The windows after the last tokens go to state_out: a new tensor by default or, with slots, `state` itself; it may
    be `state`, and must not overlap it otherwise."""
    with _On(x, stream) as s:
        if state_out is None:
            if slots is not None:
                state_out = state
            else:
                S = x.shape[0] if offsets is None else offsets.shape[0] - 1
                state_out = torch.empty((S, w.shape[-1] - 1, x.shape[-1]), dtype=x.dtype, device=x.device)
        packed, S, a = _conv_args(x, w, b, silu, offsets, slots, state, state_out)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        a.y = _View(*_view(y, packed))
        _check(_lib().seq_causal_conv(ctypes.byref(a), s), "causal_conv")
    return y, state_out


def causal_conv_step(x, state, w, b=None, silu=False, slots=None, state_out=None, stream=None):
    """causal_conv for one token of each sequence: x [S, D] -> y [S, D].  The new windows go to state_out, by default
    `state` itself."""
    with _On(x, stream) as s:
        if x.dim() != 2:
            raise ValueError("x must be [S, D], got shape %s" % (tuple(x.shape),))
        packed, S, a = _conv_args(x.unsqueeze(1), w, b, silu, None, slots, state, state if state_out is None else state_out)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        a.y = _View(y.data_ptr(), y.stride(0), 0)
        _check(_lib().seq_causal_conv_step(ctypes.byref(a), s), "causal_conv_step")
    return y


def causal_conv_grad(dy, x, w, b=None, silu=False, offsets=None, slots=None, state=None, dstate_out=None, stream=None):
    """Gradients of causal_conv: (dx, dw, db, dstate), db None without b and dstate [S, W - 1, D] None without state.
    dstate_out [S, W - 1, D]: the gradient of the outgoing windows."""
    with _On(x, stream) as s:
        packed, S, a = _conv_args(x, w, b, silu, offsets, slots, state, None)
        D, W = w.shape
        _like(dy, "dy", x.shape, x.dtype, x.device)
        if dstate_out is not None:
            _dense(dstate_out, "dstate_out", (S, W - 1, D), x.dtype, x.device)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty((D, W), dtype=torch.float32, device=x.device)
        db = torch.empty((D,), dtype=torch.float32, device=x.device) if b is not None else None
        dstate = torch.empty((S, W - 1, D), dtype=x.dtype, device=x.device) if state is not None else None
        g = ConvGradArgs(a, _view(dy, packed), dstate_out.data_ptr() if dstate_out is not None else 0, _view(dx, packed),
                         dw.data_ptr(), db.data_ptr() if b is not None else 0,
                         dstate.data_ptr() if state is not None else 0)
        n = _bytes("seq_causal_conv_grad_workspace", g)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        _check(_lib().seq_causal_conv_grad(ctypes.byref(g), ws.data_ptr(), n, s), "causal_conv_grad")
    return dx, dw, db, dstate


# ---------------------------------------------------------------------------------------------------------- scan

def _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, slots, state, state_out, max_len):
    packed, S, L = _sequences(u, offsets, "u")
    D = u.shape[-1]
    lead = 1 if packed else 2
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError("A must be [%d, states], got shape %s" % (D, tuple(A.shape)))
    N = A.shape[1]
    if B.dim() != lead + 2 or B.shape[-2] < 1 or D % B.shape[-2]:
        raise ValueError("B and C must be [..., groups, states] with groups dividing %d, got %s" % (D, tuple(B.shape)))
    G = B.shape[-2]
    _like(u, "u", u.shape, u.dtype, u.device)
    for t, name in ((delta, "delta"), (z, "z")):
        if t is not None:
            _like(t, name, u.shape, u.dtype, u.device)
    for t, name in ((B, "B"), (C, "C")):
        _like(t, name, u.shape[:-1] + (G, N), u.dtype, u.device)
    slot_ptr, P = _pool(state, state_out, slots, S, (D, N), torch.float32, u.device)
    tokens = (S, L, _index(offsets, "offsets", S + 1, u.device), slot_ptr, P)
    a = ScanArgs(tokens, D, G, N, _dtype_code(u), bool(softplus), 0, max_len or 0, _view(u, packed), _view(delta, packed),
                 _view(z, packed) if z is not None else (0, 0, 0), _view(B, packed), _view(C, packed), B.stride(-2),
                 C.stride(-2), _param(A, "A", (D, N), u.device), _param(skip, "skip", (D,), u.device),
                 _param(delta_bias, "delta_bias", (D,), u.device), *_state(state), *_state(state_out))
    return packed, S, a


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
    with _On(u, stream) as s:
        if state_out is None:
            if slots is not None:
                state_out = state
            else:
                S = u.shape[0] if offsets is None else offsets.shape[0] - 1
                state_out = torch.empty((S,) + tuple(A.shape), dtype=torch.float32, device=u.device)
        packed, S, a = _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, slots, state, state_out,
                                  max_len)
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        a.y = _View(*_view(y, packed))
        saved = None
        if save:
            saved = torch.empty(_bytes("seq_selective_scan_save", a) // 4, dtype=torch.float32, device=u.device)
            a.save = saved.data_ptr()
        n = _bytes("seq_selective_scan_workspace", a)
        ws = torch.empty(n, dtype=torch.uint8, device=u.device) if n else None
        _check(_lib().seq_selective_scan(ctypes.byref(a), ws.data_ptr() if n else 0, n, s), "selective_scan")
    return y, state_out, saved


def selective_scan_step(u, delta, A, B, C, state, skip=None, z=None, delta_bias=None, softplus=False, slots=None,
                        state_out=None, stream=None):
    """selective_scan for one token of each sequence: u, delta, z [S, D], B, C [S, G, N] -> y [S, D].  The new states
    go to state_out, by default `state` itself."""
    with _On(u, stream) as s:
        if u.dim() != 2:
            raise ValueError("u must be [S, D], got shape %s" % (tuple(u.shape),))
        packed, S, a = _scan_args(u.unsqueeze(1), delta.unsqueeze(1), A, B.unsqueeze(1), C.unsqueeze(1), skip,
                                  z.unsqueeze(1) if z is not None else None, delta_bias, softplus, None, slots, state,
                                  state if state_out is None else state_out, 1)
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        a.y = _View(y.data_ptr(), y.stride(0), 0)
        _check(_lib().seq_selective_scan_step(ctypes.byref(a), s), "selective_scan_step")
    return y


def selective_scan_grad(dy, u, delta, A, B, C, saved, skip=None, z=None, delta_bias=None, softplus=False, offsets=None,
                        max_len=None, slots=None, state=None, dstate_out=None, stream=None):
    """Gradients of selective_scan, from dy, its inputs and its `saved`: a ScanGrads tuple.  dstate_out float32 [S, D,
    N]: the gradient of the final states; dstate is that of the first ones, in the order of the sequences."""
    with _On(u, stream) as s:
        packed, S, a = _scan_args(u, delta, A, B, C, skip, z, delta_bias, softplus, offsets, slots, state, None, max_len)
        D, N = A.shape
        _like(dy, "dy", u.shape, u.dtype, u.device)
        if dstate_out is not None:
            _dense(dstate_out, "dstate_out", (S, D, N), torch.float32, u.device)
        need = _bytes("seq_selective_scan_save", a) // 4
        _dense(saved, "saved", (need,), torch.float32, u.device)
        a.save = saved.data_ptr()

        def empty(shape, dtype, wanted=True):
            return torch.empty(shape, dtype=dtype, device=u.device) if wanted else None

        f32 = torch.float32
        out = ScanGrads(du=empty(u.shape, u.dtype), ddelta=empty(u.shape, u.dtype), dA=empty((D, N), f32),
                        dB=empty(B.shape, u.dtype), dC=empty(B.shape, u.dtype), dskip=empty((D,), f32, skip is not None),
                        dz=empty(u.shape, u.dtype, z is not None),
                        ddelta_bias=empty((D,), f32, delta_bias is not None),
                        dstate=empty((S, D, N), f32, state is not None))
        g = ScanGradArgs(a, _view(dy, packed), dstate_out.data_ptr() if dstate_out is not None else 0,
                         *(t.data_ptr() if t is not None else 0 for t in
                           (out.du, out.ddelta, out.dz, out.dB, out.dC, out.dA, out.dskip, out.ddelta_bias, out.dstate)))
        n = _bytes("seq_selective_scan_grad_workspace", g)
        ws = torch.empty(n, dtype=torch.uint8, device=u.device)
        _check(_lib().seq_selective_scan_grad(ctypes.byref(g), ws.data_ptr(), n, s), "selective_scan_grad")
    return out

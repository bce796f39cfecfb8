"""The sequence operators in 64 bits on the CPU, token by token as their definitions read, differentiable by autograd,
and the tolerances of the GPU tests."""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24          # a rounding in 32 bits, relative
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def close(got, ref, dtype, c, what="", scale=None):
    """|got - ref| <= one rounding of the output + c roundings in 32 bits of `scale` (the magnitude that a sum's terms
    reach; by default the largest value of the tensor), smallest normal number of the type aside."""
    got = got.detach().double().cpu()
    ref = ref.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    top = ref[torch.isfinite(ref)].abs().max() if torch.isfinite(ref).any() else torch.tensor(0.0)
    scale = top if scale is None else scale
    tol = half_step(dtype) * ref.abs() + c * EPS32 * scale + torch.finfo(dtype).tiny
    bad = ~((got - ref).abs() <= tol) & ~((got == ref) | (got.isnan() & ref.isnan()))
    assert not bad.any(), "%s: %d of %d wrong, worst %.3e over its tolerance, at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() - tol)[bad].max()), bad.nonzero()[0].tolist())


def norm(x, residual, w, eps):
    """(y, h, r); x, residual already hold their type's values, h is rounded to x's type."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    hd = h.double()
    r = (hd.pow(2).mean(-1) + eps).rsqrt()
    return hd * r[..., None] * w.double(), h, r


def silu(v):
    return v * torch.sigmoid(v)


def ranges(offsets, x):
    """[(batch, first, end)] of the sequences of [S, L, ...] or [T, ...] rows."""
    if offsets is None:
        return [((s,), 0, x.shape[1]) for s in range(x.shape[0])]
    return [((), offsets[s], offsets[s + 1]) for s in range(len(offsets) - 1)]


def rows_of(t, b, lo, hi):
    return (t[b[0]] if b else t)[lo:hi]


def conv(x, w, b, act, offsets, state):
    """(y, windows); state [S, W - 1, D] by sequence or None.  Rows outside every sequence give zeros."""
    W = w.shape[1]
    parts, windows = {}, []
    for s, (bi, lo, hi) in enumerate(ranges(offsets, x)):
        head = state[s] if state is not None else x.new_zeros(W - 1, x.shape[-1])
        line = torch.cat([head, rows_of(x, bi, lo, hi)])
        p = sum(line[k:k + hi - lo] * w[:, k] for k in range(W)) + (b if b is not None else 0)
        parts[s] = silu(p) if act else p
        windows.append(line[hi - lo:])
    return join(parts, x, offsets), torch.stack(windows)


def join(parts, x, offsets):
    if offsets is None:
        return torch.stack([parts[s] for s in range(x.shape[0])])
    out = [parts[s] for s in sorted(parts)] + [x.new_zeros(x.shape[0] - offsets[-1], x.shape[1])]
    return torch.cat(out)


def scan(u, delta, A, B, C, skip, z, bias, softplus, offsets, state):
    """(y, states [S, D, N])."""
    D, N = A.shape
    G = B.shape[-2]
    chan = torch.arange(D) // (D // G)
    dt = delta + (bias if bias is not None else 0)
    if softplus:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    parts, finals = {}, []
    for s, (bi, lo, hi) in enumerate(ranges(offsets, u)):
        h = state[s] if state is not None else u.new_zeros(D, N)
        us, ds, Bs, Cs = (rows_of(t, bi, lo, hi) for t in (u, dt, B, C))
        ys = []
        for t in range(hi - lo):
            h = torch.exp(ds[t][:, None] * A) * h + (ds[t] * us[t])[:, None] * Bs[t][chan]
            o = (h * Cs[t][chan]).sum(-1)
            ys.append(o + (skip * us[t] if skip is not None else 0))
        y = torch.stack(ys) if ys else u.new_zeros(0, D)
        if z is not None:
            y = y * silu(rows_of(z, bi, lo, hi))
        parts[s] = y
        finals.append(h)
    return join(parts, u, offsets), torch.stack(finals)


def grads(outputs, seeds, inputs):
    """Gradients of sum(output * seed) with respect to inputs (None among them stay None)."""
    loss = sum((o * s).sum() for o, s in zip(outputs, seeds) if s is not None)
    live = [t for t in inputs if t is not None]
    got = iter(torch.autograd.grad(loss, live, allow_unused=True))
    return [None if t is None else (lambda g: torch.zeros_like(t) if g is None else g)(next(got)) for t in inputs]


def leaf(t):
    return None if t is None else t.detach().double().cpu().requires_grad_(True)

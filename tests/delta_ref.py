"""The gated delta rule in 64 bits on the CPU, token by token as its definition reads, differentiable by autograd, and the
tolerances of its GPU tests."""
from __future__ import annotations

import torch

from sequence_ref import EPS32, half_step, ranges, rows_of


def delta(q, k, v, g, beta, scale=None, offsets=None, state=None):
    """(o, states [S, H, Dk, Dv]) of q, k [S, L, Hk, Dk], v [S, L, H, Dv], g, beta [S, L, H], or of packed rows."""
    H, Dv = v.shape[-2:]
    Hk, Dk = q.shape[-2:]
    scale = Dk ** -0.5 if scale is None else scale
    head = torch.arange(H) // (H // Hk)
    outs, finals = [], []
    for s, (b, lo, hi) in enumerate(ranges(offsets, v)):
        S = state[s] if state is not None else v.new_zeros(H, Dk, Dv)
        qs, ks, vs, gs, bs = (rows_of(t, b, lo, hi) for t in (q, k, v, g, beta))
        parts = []
        for t in range(hi - lo):
            S = S * torch.exp(gs[t])[:, None, None]
            kt = ks[t][head]
            err = vs[t] - (kt[:, :, None] * S).sum(1)
            S = S + kt[:, :, None] * (bs[t][:, None] * err)[:, None, :]
            parts.append(scale * (qs[t][head][:, :, None] * S).sum(1))
        outs.append(torch.stack(parts) if parts else v.new_zeros(0, H, Dv))
        finals.append(S)
    if offsets is None:
        return torch.stack(outs), torch.stack(finals)
    return torch.cat(outs + [v.new_zeros(v.shape[0] - offsets[-1], H, Dv)]), torch.stack(finals)


def dg_scale(o, v, dv, do, dg):
    """What the terms of dg reach.  Every o is linear in its q, so q . dq = do . o; S^T k = v - z with the error z, so that
    the gates' own part of a token is k . reads = -dv . (v - z) and beta dbeta = dv . z, and together they are -dv . v.  A
    chunk's dg adds up to 64 of do . o - dv . v, whose roundings add by their squares (8), beside one whole sum dg."""
    o, v, dv, do = (t.detach().double() for t in (o, v, dv, do))
    if v.numel() == 0:
        return 0.0
    return 8 * float((do.norm(dim=-1) * o.norm(dim=-1) + 2 * dv.norm(dim=-1) * v.norm(dim=-1)).max()) + float(dg.abs().max())


def close(got, ref, dtype, roundings, chain, what, scale=None):
    """Each element: one rounding of the output and `roundings` of 32 bits, one after the other, of the tensor's largest
    value (for sums whose terms reach four times it) or of `scale`.  The whole: as errors of independent roundings add by
    their squares, sqrt(roundings) of them relative to the tensor's norm, eight times for the `chain` of steps that pass
    them on."""
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    assert bool(torch.isfinite(got).all()), what
    off, top = (got - ref).abs(), float(ref.abs().max()) if scale is None else scale
    tol = half_step(dtype) * ref.abs() + 4 * roundings * EPS32 * top + torch.finfo(dtype).tiny
    assert bool((off <= tol).all()), "%s: %d of %d wrong, worst %.3e, at %s" % (
        what, int((off > tol).sum()), off.numel(), float((off - tol).max()), (off > tol).nonzero()[0].tolist())
    norm = float(ref.norm()) if scale is None else scale * off.numel() ** 0.5
    whole = half_step(dtype) * float(ref.norm()) + 8 * (roundings * chain) ** 0.5 * EPS32 * norm
    assert float(off.norm()) <= whole + torch.finfo(dtype).tiny * off.numel() ** 0.5, (what, float(off.norm()), whole)

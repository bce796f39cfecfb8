"""The gated delta rule's chunk form with the arithmetic of its kernels, on the CPU: operands of every product cut to
pieces of bf16, products and sums in 32 bits.  With as many pieces as the kernels take (three: 24 bits) its errors against
the definition in 64 bits say how far off results in 32 bits are, from which the bounds here are derived; with two (16
bits) they say what these bounds have to catch."""
from __future__ import annotations

import torch

CHUNK = 64


def cut(x, n):
    """n bf16 numbers, as floats, whose sum is x to 8 n bits."""
    out = []
    for _ in range(n):
        out.append(x.bfloat16().float())
        x = x - out[-1]
    return out


def product(a, b, n):
    """a @ b of the pieces' products above 2^-8n of the whole, the small ones first."""
    pa, pb = cut(a, n), cut(b, n)
    return sum(pa[i] @ pb[s - i] for s in range(n - 1, -1, -1) for i in range(s + 1))


def chunked(q, k, v, g, beta, state=None, do=None, dlast=None, pieces=3, out_pieces=3):
    """(o, state) of q, k [S, L, Hk, Dk], v [S, L, H, Dv], g, beta [S, L, H] in 32 bits, not rounded to their type; with do
    also (dq, dk, dv, dg, dbeta, dstate)."""
    S, L, H, Dv = v.shape
    Hk, Dk = q.shape[-2:]
    group, scale, dt = H // Hk, Dk ** -0.5, q.dtype
    chunks = -(-L // CHUNK)

    def lay(t):          # [S, H, chunks, CHUNK, ...], zeros behind the end
        out = t.new_zeros((S, chunks * CHUNK) + t.shape[2:])
        out[:, :L] = t
        return out.movedim(2, 1).unflatten(2, (chunks, CHUNK))

    def back(t):
        return t.flatten(2, 3)[:, :, :L].movedim(1, 2)

    q, k = (lay(t.float().repeat_interleave(group, 2)) for t in (q, k))
    v, g, beta = lay(v.float()), lay(g.double()), lay(beta)
    G = g.cumsum(-1)
    e = torch.exp((G[..., :, None] - G[..., None, :]).tril()).float().tril()
    first, last = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    b = beta[..., None]
    M = (product(k, k.mT, 3) * e * beta[..., None, :]).tril(-1)
    eye = torch.eye(CHUNK)
    T = torch.linalg.solve_triangular(eye + M, eye.expand_as(M), upper=False, unitriangular=True)
    P = scale * product(q, k.mT, 3) * e * beta[..., None, :]
    at = state.float() if state is not None else v.new_zeros(S, H, Dk, Dv)
    states, o, z = [at], torch.empty_like(v), torch.empty_like(v)
    for n in range(chunks):
        x = v[:, :, n] - first[:, :, n] * product(k[:, :, n], at, pieces)
        z[:, :, n] = product(T[:, :, n], x, pieces)
        o[:, :, n] = scale * first[:, :, n] * product(q[:, :, n], at, out_pieces) + product(P[:, :, n], z[:, :, n], out_pieces)
        at = first[:, :, n, -1:] * at + product(k[:, :, n].mT, last[:, :, n] * b[:, :, n] * z[:, :, n], pieces)
        states.append(at)
    if do is None:
        return back(o), at
    do = lay(do.float())
    dS = dlast.float() if dlast is not None else torch.zeros_like(at)
    dS_of, dx, tail = [None] * chunks, torch.empty_like(v), []
    for n in range(chunks - 1, -1, -1):
        dS_of[n] = dS
        tail.insert(0, (dS * states[n + 1]).sum((-1, -2)))
        dz = b[:, :, n] * last[:, :, n] * product(k[:, :, n], dS, pieces) + product(P[:, :, n].mT, do[:, :, n], pieces)
        dx[:, :, n] = product(T[:, :, n].mT, dz, pieces)
        dS = (first[:, :, n, -1:] * dS + product(q[:, :, n].mT, scale * first[:, :, n] * do[:, :, n], pieces)
              - product(k[:, :, n].mT, first[:, :, n] * dx[:, :, n], pieces))
    S_in, dS_out = torch.stack(states[:-1], 2).mT, torch.stack(dS_of, 2).mT
    E = scale * product(do, z.mT, pieces) * e
    R = product(dx, z.mT, pieces) * e.tril(-1)
    bj = beta[..., None, :]
    dq = scale * first * product(do, S_in, pieces) + product(E * bj, k, pieces)
    reads = -first * product(dx, S_in, pieces) - product(R * bj, k, pieces)
    w = last * product(z, dS_out, pieces) + product(E.mT, q, pieces) - product(R.mT, k, pieces)
    dbeta = (k * w).sum(-1)
    dG = ((q * dq + k * reads).sum(-1) - beta * dbeta).double()
    dg = (dG.flip(-1).cumsum(-1).flip(-1) + torch.stack(tail, 2)[..., None]).float()

    def grouped(t):
        return back(t).unflatten(2, (Hk, group)).sum(3)

    return (back(o), at), (grouped(dq), grouped(reads + b * w), back(dx), back(dg), back(dbeta), dS)


# ---- cases and bounds -------------------------------------------------------------------------------------------------

NAMES = ("o", "state", "dq", "dk", "dv", "dg", "dbeta", "dstate")
# lengths, key heads, heads, Dk, Dv, keys and gates
CASES = [
    ((64,), 1, 1, 16, 16, "usual"), ((65, 65), 1, 2, 64, 32, "usual"), ((200,), 1, 2, 128, 128, "usual"),
    ((130, 130), 1, 4, 128, 64, "usual"), ((65, 0, 130), 2, 4, 64, 64, "usual"), ((129, 1, 66), 1, 2, 128, 32, "usual"),
    ((129,), 1, 4, 256, 64, "usual"), ((70,), 1, 1, 200, 130, "usual"), ((130, 130), 2, 4, 72, 41, "usual"),
    ((300,), 1, 2, 64, 32, "alike"), ((257,), 1, 1, 128, 64, "alike"), ((4096,), 1, 1, 16, 16, "slow"),
    ((2500,), 1, 2, 64, 32, "slow"), ((130, 65), 1, 2, 64, 32, "growing")]


def unit(t):
    return t / t.norm(dim=-1, keepdim=True)


def inputs(case, dt):
    """Packed rows q, k, v, g, beta, state, do, dlast on the CPU in their types.  alike: keys a tenth apart and beta next to
    one, so that each token's correction takes back most of the last one's.  slow: a memory of thousands of tokens.  growing: states
    that grow tenfold in some thirty tokens."""
    lens, Hk, H, Dk, Dv, kind = case
    rand = torch.Generator().manual_seed(sum(lens) * 31 + Dk * 7 + Dv)
    r = lambda *s: torch.randn(*s, generator=rand)  # noqa: E731
    T, S = sum(lens), len(lens)
    q, k, v, g, b = r(T, Hk, Dk), r(T, Hk, Dk), r(T, H, Dv), r(T, H), r(T, H)
    if kind == "alike":
        k = k[:1] / k[:1].norm(dim=-1, keepdim=True) + 0.1 * unit(k)
    g = -torch.nn.functional.softplus(g - 2) * torch.linspace(0.1, 4, H)
    beta = torch.sigmoid(b + 4) if kind == "alike" else torch.sigmoid(b)
    if kind == "slow":
        g, beta = g * 1e-3, beta * 0.01
    if kind == "growing":
        g = 0.05 - 0.05 * g.clamp(min=-1)
    return ([unit(q).to(dt), unit(k).to(dt), v.to(dt), g, beta, 0.3 * r(S, H, Dk, Dv)], r(T, H, Dv).to(dt),
            0.3 * r(S, H, Dk, Dv))


def offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def emulated(case, ins, do, dlast, pieces, out_pieces):
    """{name: 32-bit result} of the packed rows, sequence by sequence."""
    *rows, state = ins
    parts = []
    for s, (lo, hi) in enumerate(zip(offsets(case[0]), offsets(case[0])[1:])):
        if lo == hi:
            parts.append([t[lo:hi].float() for t in (rows[2],)] + [state[s]] + [t[lo:hi].float() for t in rows] + [dlast[s]])
            continue
        fwd, grad = chunked(*(t[None, lo:hi] for t in rows), state=state[s:s + 1], do=do[None, lo:hi], dlast=dlast[s:s + 1],
                            pieces=pieces, out_pieces=out_pieces)
        parts.append([t[0] for t in (*fwd, *grad)])
    join = [torch.stack if n in ("state", "dstate") else torch.cat for n in NAMES]
    return {n: f([p[i] for p in parts]) for i, (n, f) in enumerate(zip(NAMES, join))}


def sizes(case, ins, do, want):
    """What each output's error is measured against: its norm, and for dg, a sum of differences, that of the terms: each
    token adds do . o and dv . v (every o is linear in its q; beta dbeta - k . reads = dv . v), and dg at a token takes those
    of the chunk from there on."""
    out = {n: float(t.norm()) for n, t in want.items()}
    o, v, dv, d = want["o"], ins[2].double(), want["dv"], do.double()
    terms, total = ((d * o).pow(2).sum(-1) + (dv * v).pow(2).sum(-1)), 0.0
    for lo, hi in zip(offsets(case[0]), offsets(case[0])[1:]):
        for a in range(lo, hi, CHUNK):
            total += float(terms[a:min(a + CHUNK, hi)].flip(0).cumsum(0).sum())
    out["dg"] = total ** 0.5 + out["dg"]
    return out


def errors(got, want, size):
    return {n: float((got[n].detach().double().cpu() - want[n]).norm()) / size[n] for n in want}


def neighbours(got, ref):
    """Elements that are not the 64-bit result rounded to their type."""
    return int((got.detach().cpu() != ref.to(got.dtype)).sum())


def expected_neighbours(got32, ref, dtype):
    """How many elements an error of such sizes takes over a border between two numbers of dtype: each its error over the
    distance of two such borders."""
    step = torch.finfo(dtype).eps * 2.0 ** torch.floor(torch.log2(ref.abs().clamp(min=torch.finfo(dtype).tiny)))
    return float(((got32.double() - ref).abs() / step).clamp(max=1).sum())


def error_bounds(measured):
    """Four times what the emulation of three pieces measures: the kernels add the same numbers in other orders, and their
    exponentials are off by two roundings in place of one.  dg's error is mostly that of a few sums, which may come out
    small by chance: at least five roundings."""
    return {n: 4 * max(e, 5 * 2.0 ** -24 if n == "dg" else 2.0 ** -24) for n, e in measured.items()}


def neighbour_bound(expected):
    """Errors of up to four times the size, and four deviations of a count of independent events; four where hardly any are
    expected."""
    return 4 * expected + 4 * (4 * expected) ** 0.5 + 4


def reference(case, ins, do, dlast):
    """{name: 64-bit result}: the definition, token by token, and autograd."""
    import delta_ref
    from sequence_ref import grads, leaf
    leaves = [leaf(t) for t in ins]
    o, state = delta_ref.delta(*leaves[:5], offsets=offsets(case[0]), state=leaves[5])
    return {n: t.detach() for n, t in zip(NAMES, (o, state, *grads((o, state), (do.double(), dlast.double()), leaves)))}

"""The gated delta rule on the GPU against its definition in 64 bits (delta_ref).

Tolerances: a state passes, each chunk of 64 tokens, through sums over the key's dimension (K S), over the chunk (Z) and
over the chunk again (K^T Z), whose numbers are held to 24 bits: at most Dk + 128 roundings and some 50 of the pieces, the
decays (8) and the small system's solution.  Its gradient passes through that chain twice and through sums over Dv besides;
the chain of chunks multiplies them by its length.  dg is a sum of differences (delta_ref.dg_scale)."""
import pytest
import torch

import delta_ref
import sequence_ref as ref
from gpu_util import log
from sequence_ref import DT, leaf
from test_gpu_sequence import gen

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def iga():
    import implicit_gemm_amd
    return implicit_gemm_amd


def unit(t):
    return t / t.norm(dim=-1, keepdim=True)


def make(seed, shape, Hk, H, Dk, Dv, dt):
    """q, k, v, g, beta on the CPU in their types."""
    rand = gen(seed)
    q, k = unit(rand(*shape, Hk, Dk)).to(dt), unit(rand(*shape, Hk, Dk)).to(dt)
    g = -torch.nn.functional.softplus(rand(*shape, H) - 2) * torch.linspace(0.1, 4, H)
    return q, k, rand(*shape, H, Dv).to(dt), g, torch.sigmoid(rand(*shape, H))


def parts_of_a_row(q, k, v):
    """The same values as parts of one wider projection, behind an odd number of other columns."""
    flat = [t.flatten(-2) for t in (q, k, v)]
    pad = torch.full(v.shape[:-2] + (3,), 7.0, dtype=v.dtype)
    wide = torch.cat([pad] + flat, -1).cuda()
    at, out = 3, []
    for t, f in zip((q, k, v), flat):
        out.append(wide[..., at:at + f.shape[-1]].unflatten(-1, t.shape[-2:]))
        at += f.shape[-1]
    return out


def roundings(Dk, longest):
    return (Dk + 190) * max(1, -(-longest // 64)), max(1, -(-longest // 64))


PACKED = [0, 1, 1, 66, 130, 258]
CASES = [  # offsets or (S, L), tail, Hk, H, Dk, Dv
    ((2, 1), 0, 1, 1, 1, 1), ((1, 64), 0, 1, 2, 16, 16), ((2, 65), 0, 2, 2, 64, 32), ((1, 200), 0, 1, 1, 128, 128),
    ((2, 63), 0, 3, 6, 72, 41), ((1, 130), 0, 2, 4, 100, 17), ((1, 129), 0, 1, 2, 256, 64), ((1, 70), 0, 1, 1, 200, 130),
    (PACKED, 0, 2, 2, 64, 48), (PACKED, 70, 1, 3, 128, 33), (PACKED, 1, 2, 4, 33, 128), ([0, 0], 20, 1, 1, 64, 16),
    ([0, 0, 5], 0, 1, 1, 8, 300), ((1, 0), 0, 1, 2, 64, 64), ([0, 64, 192], 0, 1, 3, 130, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("rows,tail,Hk,H,Dk,Dv", CASES)
def test_delta_and_gradient(iga, rows, tail, Hk, H, Dk, Dv, carried, dtype):
    log("delta", rows, tail, Hk, H, Dk, Dv, carried, dtype)
    dt = DT[dtype]
    packed = isinstance(rows, list)
    shape = (rows[-1] + tail,) if packed else rows
    S = len(rows) - 1 if packed else rows[0]
    longest = max(b - a for a, b in zip(rows, rows[1:])) if packed else rows[1]
    q, k, v, g, beta = make(Dk * 7 + Dv, shape, Hk, H, Dk, Dv, dt)
    rand = gen(Dk + Dv)
    do = rand(*shape, H, Dv).to(dt)
    P = S + 2
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(Dk))[:S].int()
    pool = rand(P, H, Dk, Dv, std=0.3)
    state = pool[slots.long()] if carried else None
    dlast = rand(S, H, Dk, Dv, std=0.3) if carried else None
    off = torch.tensor(rows, dtype=torch.int32).cuda() if packed else None
    qd, kd, vd = parts_of_a_row(q, k, v)
    gd, bd = g.cuda(), torch.stack([beta, beta], -1).flatten(-2).cuda()[..., :H] if H == 1 else beta.cuda()
    kw = dict(offsets=off)
    if carried:
        kw.update(state=pool.cuda(), slots=slots.cuda())
    out = torch.full((P, H, Dk, Dv), 5.0).cuda() if carried else None
    scale = 0.3 if Dk == 64 else None
    o, last, saved = iga.gated_delta(qd, kd, vd, gd, bd, scale=scale, save=True, state_out=out, **kw)
    leaves = [leaf(t) for t in (q, k, v, g, beta, state)]
    orr, lr = delta_ref.delta(*leaves[:5], scale=scale, offsets=rows if packed else None, state=leaves[5])
    c, chain = roundings(Dk, longest)
    delta_ref.close(o, orr, dt, c + Dk, chain, "o")
    if packed and tail:
        assert not o[rows[-1]:].any()
    if carried:
        delta_ref.close(last[slots.long().cuda()], lr, torch.float32, c, chain, "state")
        untouched = torch.ones(P, dtype=torch.bool)
        untouched[slots.long()] = False
        assert bool((last[untouched.cuda()] == 5).all())
        inplace = pool.cuda()
        o2, last2, none = iga.gated_delta(qd, kd, vd, gd, bd, scale=scale, offsets=off, state=inplace, slots=slots.cuda())
        assert none is None and last2 is inplace and torch.equal(o2, o)
        assert torch.equal(last2[slots.long().cuda()], last[slots.long().cuda()])
    else:
        delta_ref.close(last, lr, torch.float32, c, chain, "state")
        assert torch.equal(iga.gated_delta(qd, kd, vd, gd, bd, scale=scale, offsets=off)[0], o)
    d = iga.gated_delta_grad(do.cuda(), qd, kd, vd, gd, bd, saved, scale=scale, offsets=off,
                             dstate_out=dlast.cuda() if carried else None,
                             **(dict(state=pool.cuda(), slots=slots.cuda()) if carried else {}))
    grads = ref.grads((orr, lr), (do.double(), dlast.double() if carried else None), leaves) if orr.requires_grad or carried else \
        [torch.zeros_like(t) if t is not None else None for t in leaves]
    c = 2 * c + Dv + 64
    for name, got, want, t in (("dq", d.dq, grads[0], dt), ("dk", d.dk, grads[1], dt), ("dv", d.dv, grads[2], dt),
                               ("dg", d.dg, grads[3], torch.float32), ("dbeta", d.dbeta, grads[4], torch.float32)):
        top = delta_ref.dg_scale(orr, v, grads[2], do, grads[3]) if name == "dg" else None
        delta_ref.close(got, want, t, c * (H // Hk if name in ("dq", "dk") else 1), chain, name, scale=top)
        if packed and tail:
            assert not got[rows[-1]:].any(), name
    assert (d.dstate is None) == (not carried)
    if carried:
        delta_ref.close(d.dstate, grads[5], torch.float32, c, chain, "dstate")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S,Hk,H,Dk,Dv", [(1, 1, 1, 1, 1), (3, 2, 2, 64, 64), (5, 3, 6, 72, 41), (2, 1, 2, 128, 128),
                                          (2, 2, 2, 256, 256), (4, 1, 4, 17, 130), (70, 1, 1, 200, 5), (1, 1, 1, 64, 1024)])
def test_step(iga, S, Hk, H, Dk, Dv, dtype):
    log("delta step", S, Hk, H, Dk, Dv, dtype)
    dt = DT[dtype]
    q, k, v, g, beta = make(S + Dk, (S,), Hk, H, Dk, Dv, dt)
    if S > 2:
        g[1] = -float("inf")
    P = S + 1
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(Dk))[:S].int()
    if S > 3:
        slots[2], slots[3] = -1, P                      # rows of padding
    pool = gen(3)(P, H, Dk, Dv)
    live = (slots >= 0) & (slots < P)
    state = torch.where(live[:, None, None, None], pool[slots.long().clamp(0, P - 1)], torch.zeros(1))
    o_ref, s_ref = delta_ref.delta(*(t[:, None].double() for t in (q, k, v, g, beta)), state=state.double())
    qd, kd, vd = parts_of_a_row(q, k, v)
    inplace = pool.cuda()
    o = iga.gated_delta_step(qd, kd, vd, g.cuda(), beta.cuda(), inplace, slots=slots.cuda())
    delta_ref.close(o, o_ref[:, 0], dt, Dk + 16, 1, "o")
    want = pool.clone().double()
    want[slots[live].long()] = s_ref[live]
    delta_ref.close(inplace, want, torch.float32, Dk + 16, 1, "state")
    free = torch.ones(P, dtype=torch.bool)
    free[slots[live].long()] = False
    assert torch.equal(inplace.cpu()[free], pool[free])
    elsewhere = torch.full_like(inplace, 5.0)
    o2 = iga.gated_delta_step(qd, kd, vd, g.cuda(), beta.cuda(), pool.cuda(), slots=slots.cuda(), state_out=elsewhere)
    assert torch.equal(o2, o) and torch.equal(elsewhere.cpu()[~free], inplace.cpu()[~free]) and bool((elsewhere.cpu()[free] == 5).all())


def test_steps_continue_a_prompt(iga):
    """A prompt of 70 tokens and one of 69 with a step behind it end in the same state, to its rounding."""
    q, k, v, g, beta = (t.cuda() for t in make(4, (2, 70), 2, 4, 128, 64, torch.bfloat16))
    o, want, _ = iga.gated_delta(q, k, v, g, beta)
    o1, state, _ = iga.gated_delta(q[:, :69], k[:, :69], v[:, :69], g[:, :69], beta[:, :69])
    o2 = iga.gated_delta_step(q[:, 69], k[:, 69], v[:, 69], g[:, 69], beta[:, 69], state)
    c, chain = roundings(128, 70)
    delta_ref.close(state, want, torch.float32, 2 * c, chain, "state")
    assert torch.equal(o1, o[:, :69])
    delta_ref.close(o2, o[:, 69], torch.bfloat16, 2 ** 17, 1, "o")      # both are rounded: a step of bf16 apart at most
    cut, mid, _ = iga.gated_delta(q[:, :33], k[:, :33], v[:, :33], g[:, :33], beta[:, :33])
    rest, end, _ = iga.gated_delta(q[:, 33:], k[:, 33:], v[:, 33:], g[:, 33:], beta[:, 33:], state=mid, state_out=mid)
    assert end is mid
    delta_ref.close(end, want, torch.float32, 2 * c, chain, "state in two calls")


@pytest.mark.parametrize("dtype", TYPES)
def test_edges_of_the_gates(iga, dtype):
    """Decays of nothing, of everything (-inf) and of more than 32 bits hold; beta of 0, 1 and 1.5; keys and queries of
    zeros."""
    dt = DT[dtype]
    q, k, v, g, beta = make(11, (1, 150), 1, 3, 64, 32, dt)
    g[0, :, 0] = 0
    g[0, ::7, 1] = -float("inf")
    g[0, 1::3, 2] = -150.0
    g[0, 2::31, 2] = -1e30
    beta[0, ::5] = 0
    beta[0, 1::5] = 1
    beta[0, 2::15] = 1.5
    k[0, 40:43] = 0
    q[0, 50] = 0
    do = gen(2)(1, 150, 3, 32).to(dt)
    o, last, saved = iga.gated_delta(*(t.cuda() for t in (q, k, v, g, beta)), save=True)
    d = iga.gated_delta_grad(do.cuda(), *(t.cuda() for t in (q, k, v, g, beta)), saved)
    leaves = [leaf(t) for t in (q, k, v, g.clamp(min=-1e4), beta)]        # e^-10000 is zero in 64 bits as well
    orr, lr = delta_ref.delta(*leaves)
    grads = ref.grads((orr,), (do.double(),), leaves)
    c, chain = roundings(64, 150)
    delta_ref.close(o, orr, dt, c, chain, "o")
    delta_ref.close(last, lr, torch.float32, c, chain, "state")
    for name, got, want, t in zip(d._fields, d, grads, (dt, dt, dt, torch.float32, torch.float32)):
        top = delta_ref.dg_scale(orr, v, grads[2], do, grads[3]) if name == "dg" else None
        delta_ref.close(got, want, t, (2 * c + 96) * 3, chain, name, scale=top)


def test_nan_stays_in_its_sequence_and_head(iga):
    q, k, v, g, beta = make(5, (200,), 2, 2, 64, 32, torch.float32)
    off = torch.tensor([0, 70, 140, 190], dtype=torch.int32)
    v[100, 0, 3] = float("nan")
    k[200 - 5] = float("inf")                            # padding
    o, last, saved = iga.gated_delta(*(t.cuda() for t in (q, k, v, g, beta)), offsets=off.cuda(), save=True)
    assert bool(torch.isfinite(o[:70]).all()) and bool(torch.isfinite(o[140:]).all()) and not o[190:].any()
    assert bool(torch.isfinite(o[70:140, 1]).all()) and bool(o[101:140, 0, 3].isnan().all())
    assert bool(torch.isfinite(o[70:140, 0, :3]).all()) and bool(torch.isfinite(o[70:140, 0, 4:]).all())
    assert bool(torch.isfinite(last[[0, 2]]).all()) and bool(last[1, 0, :, 3].isnan().all())
    d = iga.gated_delta_grad(torch.ones_like(v).cuda(), *(t.cuda() for t in (q, k, v, g, beta)), saved, offsets=off.cuda())
    for t in d[:5]:
        assert bool(torch.isfinite(t[:70]).all()) and bool(torch.isfinite(t[140:]).all()) and bool(torch.isfinite(t[70:140, 1]).all())


def test_slots_without_a_state(iga):
    q, k, v, g, beta = (t.cuda() for t in make(6, (3, 65), 1, 2, 64, 16, torch.float32))
    pool = gen(1)(2, 2, 64, 16).cuda()
    before = pool.clone()
    o, last, _ = iga.gated_delta(q, k, v, g, beta, state=pool, slots=torch.tensor([-1, 1, 9], dtype=torch.int32).cuda())
    fresh = iga.gated_delta(q, k, v, g, beta)[0]
    assert last is pool and torch.equal(pool[0], before[0]) and not torch.equal(pool[1], before[1])
    assert torch.equal(o[0], fresh[0]) and torch.equal(o[2], fresh[2]) and not torch.equal(o[1], fresh[1])


def test_runs_repeat_bit_for_bit_on_any_stream_and_in_a_graph(iga):
    inputs = [t.cuda() for t in make(8, (2, 200), 2, 4, 128, 64, torch.bfloat16)]
    do = gen(3)(2, 200, 4, 64).to(torch.bfloat16).cuda()
    one = [t[:, 0].contiguous() for t in inputs]
    pool = gen(4)(2, 4, 128, 64).cuda()

    def step(**kw):
        o, last, saved = iga.gated_delta(*inputs, state=pool, state_out=torch.empty_like(pool), save=True, **kw)
        d = iga.gated_delta_grad(do, *inputs, saved, state=pool, dstate_out=last, **kw)
        after = torch.empty_like(pool)
        return (o, last) + tuple(d) + (iga.gated_delta_step(*one, last, state_out=after, **kw), after)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    o = iga.gated_delta(*inputs, state=pool, state_out=torch.empty_like(pool), stream=side)[0]
    side.synchronize()
    assert torch.equal(o, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        for t, n in zip(inputs, make(20 + seed, (2, 200), 2, 4, 128, 64, torch.bfloat16)):
            t.copy_(n)
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))


def test_gradient_against_differences(iga):
    """At full precision, along one direction of each input: the definition's own differences in 64 bits."""
    ins = [t.double() for t in make(9, (1, 90), 1, 2, 16, 8, torch.float32)]
    do = gen(1)(1, 90, 2, 8).double()

    def loss(*a):
        return float((delta_ref.delta(*a)[0] * do).sum())

    dev = [t.float().cuda() for t in ins]
    _, _, saved = iga.gated_delta(*dev, save=True)
    d = iga.gated_delta_grad(do.float().cuda(), *dev, saved)
    for i, got in enumerate(d[:5]):
        way = gen(30 + i)(*ins[i].shape).double()
        h = 1e-5
        more, less = ([t + s * h * way if j == i else t for j, t in enumerate(ins)] for s in (1, -1))
        want = (loss(*more) - loss(*less)) / (2 * h)
        have = float((got.double().cpu() * way).sum())
        # differences are good to h^2 of the third derivative; the sum's terms add by their squares
        tol = 1e-5 * (abs(want) + float((got.double().cpu() * way).norm()))
        assert abs(want - have) < tol, (i, want, have)


def test_many_sequences_and_rows_past_4_gib(iga):
    """16384 sequences of one to three tokens, and values that begin past 4 GiB, against parts of themselves."""
    lens = [1 + i % 3 for i in range(16384)]
    off = torch.cumsum(torch.tensor([0] + lens), 0).int()
    T = int(off[-1])
    q, k, v, g, beta = (t.cuda() for t in make(12, (T,), 1, 1, 16, 16, torch.float16))
    o, last, _ = iga.gated_delta(q, k, v, g, beta, offsets=off.cuda())
    for s in (0, 1, 8191, 16383):
        lo, hi = int(off[s]), int(off[s + 1])
        o1, l1, _ = iga.gated_delta(*(t[None, lo:hi] for t in (q, k, v, g, beta)))
        assert torch.equal(o[lo:hi], o1[0]) and torch.equal(last[s], l1[0])
    L, wide = 300, 1 << 23                               # rows of 16 MB: the second sequence begins past 4 GiB
    store = torch.zeros(2 * L, wide, dtype=torch.bfloat16, device="cuda")
    q, k, v, g, beta = (t.cuda() for t in make(13, (2, L), 1, 1, 64, 32, torch.bfloat16))
    x = store.view(2, L, wide)[..., wide - 160:]
    x[..., :64], x[..., 64:128], x[..., 128:] = q.flatten(2), k.flatten(2), v.flatten(2)
    parts = (x[..., :64].unflatten(-1, (1, 64)), x[..., 64:128].unflatten(-1, (1, 64)), x[..., 128:].unflatten(-1, (1, 32)))
    o, last, saved = iga.gated_delta(*parts, g, beta, save=True)
    want, wlast, wsaved = iga.gated_delta(q, k, v, g, beta, save=True)
    assert torch.equal(o, want) and torch.equal(last, wlast) and torch.equal(saved, wsaved)
    d, w = (iga.gated_delta_grad(want, *p, g, beta, saved) for p in (parts, (q, k, v)))
    assert all(torch.equal(a, b) for a, b in zip(d[:5], w[:5]))


def test_refusals(iga):
    q, k, v, g, beta = (t.cuda() for t in make(14, (2, 10), 2, 4, 32, 16, torch.float32))
    state = torch.zeros(2, 4, 32, 16).cuda()
    _, _, saved = iga.gated_delta(q, k, v, g, beta, save=True)
    off = torch.tensor([0, 5, 10], dtype=torch.int32).cuda()
    one = [t[:, 0] for t in (q, k, v, g, beta)]
    for bad in (lambda: iga.gated_delta(q[..., :1, :].expand(2, 10, 3, 32), k, v, g, beta), lambda: iga.gated_delta(q, k[..., :16], v, g, beta),
                lambda: iga.gated_delta(q, k, v, g.double(), beta), lambda: iga.gated_delta(q, k, v, g, beta[..., :2]),
                lambda: iga.gated_delta(q.bfloat16(), k, v, g, beta), lambda: iga.gated_delta(q, k, v.double(), g, beta),
                lambda: iga.gated_delta(q, k, v, g, beta, offsets=off), lambda: iga.gated_delta(q[0], k[0], v[0], g[0], beta[0]),
                lambda: iga.gated_delta(q, k, v, g, beta, state=state[:1]), lambda: iga.gated_delta(q, k, v, g, beta, state=state.half()),
                lambda: iga.gated_delta(q, k, v, g, beta, state=state.transpose(2, 3)),
                lambda: iga.gated_delta(q.cpu(), k, v, g, beta), lambda: iga.gated_delta(q, k, v, g.cpu(), beta),
                lambda: iga.gated_delta(q.transpose(2, 3), k, v, g, beta), lambda: iga.gated_delta_step(*one, state[:1]),
                lambda: iga.gated_delta_step(q, k, v, g, beta, state),
                lambda: iga.gated_delta_grad(v[:1], q, k, v, g, beta, saved), lambda: iga.gated_delta_grad(v, q, k, v, g, beta, saved[:-1]),
                lambda: iga.gated_delta(*(torch.zeros(1, 2, 1, 257).cuda(),) * 2, v[:1, :2, :1], g[:1, :2, :1], beta[:1, :2, :1])):
        with pytest.raises((ValueError, TypeError, iga.ConvWgradError)):
            bad()


def test_two_graphs_in_turn(iga):
    """Two captured calls of other sizes, each with a workspace of its own, replayed in turn with eager calls between."""
    def case(seed, L, H, Dk, Dv, dt):
        inputs = [t.cuda() for t in make(seed, (2, L), H, H, Dk, Dv, dt)]

        def call():
            o, last, saved = iga.gated_delta(*inputs, save=True)
            return (o, last) + tuple(iga.gated_delta_grad(o, *inputs, saved)[:5])
        return call

    calls = [case(41, 150, 2, 128, 64, torch.bfloat16), case(42, 70, 3, 72, 41, torch.float32)]
    want = [[t.clone() for t in c()] for c in calls]
    graphs, outs = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(c())
    for _ in range(3):
        for g, c, o, w in zip(graphs, calls, outs, want):
            g.replay()
            again = c()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(w, o)) and all(torch.equal(a, b) for a, b in zip(w, again))


def test_the_largest_sizes_against_parts_of_themselves(iga):
    """Columns of v are independent of each other, and so are heads: calls of the most columns and of the most heads give
    what calls of a part give."""
    q, k, v, g, beta = (t.cuda() for t in make(15, (2, 70), 1, 1, 256, 1024, torch.bfloat16))
    part = slice(992, 1024)
    o, last, saved = iga.gated_delta(q, k, v, g, beta, save=True)
    o1, last1, _ = iga.gated_delta(q, k, v[..., part].contiguous(), g, beta)
    assert torch.equal(o[..., part], o1) and torch.equal(last[..., part], last1)
    dv = iga.gated_delta_grad(o, q, k, v, g, beta, saved).dv
    _, _, saved1 = iga.gated_delta(q, k, v[..., part].contiguous(), g, beta, save=True)
    assert torch.equal(dv[..., part], iga.gated_delta_grad(o1, q, k, v[..., part].contiguous(), g, beta, saved1).dv)
    one = [t[:, 0].contiguous() for t in (q, k, v, g, beta)]
    a, b = last.clone(), last[..., part].contiguous()
    y = iga.gated_delta_step(*one, a)
    one[2] = one[2][..., part].contiguous()
    # Up to 64 columns go to other teams of lanes, which add the 256 products of k S in another order: each order is off by
    # at most 256 half steps of the sum of their sizes, the sums' w then enters the state times k, and the state's own two
    # operations and w's three leave a half step of what they make each, on both sides.  o is one rounding to bf16 of sums
    # of 256 such elements: two half steps of the largest and that.
    y1 = iga.gated_delta_step(*one, b)
    before, half = last[..., part].double(), 2.0 ** -24
    k64 = one[1].double().abs()[..., None]                                     # [S, 1, Dk, 1], as the state
    tol = 512 * half * k64 * (k64 * before.abs()).sum(-2, keepdim=True) + 16 * half * (b.double().abs() + before.abs())
    assert bool(((a[..., part].double() - b.double()).abs() <= tol).all())
    assert bool(((y1.double() - y[..., part].double()).abs() <= (2.0 ** -7 + 2.0 ** -12) * y.double().abs().max()).all())
    H = 65536
    q, k, v, g, beta = (t.cuda() for t in make(16, (1, 3), H, H, 2, 4, torch.float32))
    o, last, saved = iga.gated_delta(q, k, v, g, beta, save=True)
    d = iga.gated_delta_grad(o, q, k, v, g, beta, saved)
    few = [t[:, :, -5:] for t in (q, k, v, g, beta)]
    o1, last1, saved1 = iga.gated_delta(*few, save=True)
    d1 = iga.gated_delta_grad(o1, *few, saved1)
    assert torch.equal(o[:, :, -5:], o1) and torch.equal(last[:, -5:], last1)
    assert all(torch.equal(a[:, :, -5:], b) for a, b in zip(d[:5], d1[:5]))


# ---------------------------------------------------------------------------------------------------- as a model's layer

@pytest.fixture(scope="module")
def layer_module():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_layer.py")
    spec = importlib.util.spec_from_file_location("delta_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes", [dict(Hk=2, H=4, Dk=64, Dv=64), dict(Hk=1, H=3, Dk=40, Dv=24)])
def test_layer_by_tokens_matches_prompts(layer_module, sizes, dtype):
    """The delta rule's output is linear in queries, keys and values each, which three roundings to the element type
    precede (projection, convolution, norm), and three follow (the rule's, the heads' norm's, the output's): 3 * 3 + 3
    half steps on either side, 24 of the largest output in all, and the matrix products between them sum in other
    orders: thirty-two."""
    layer = layer_module.Layer(96, dtype=DT[dtype], seed=3, **sizes)
    off = layer_module.steps_against_prompt(layer, [130, 5, 33, 17])
    assert off <= max(32 * ref.half_step(DT[dtype]), 1e-5)


def test_layer_gradient_against_difference(layer_module):
    """Central differences of a float32 loss: the step's square and the losses' rounding (2^-24 of their terms over the
    step) leave about a thousandth."""
    slope, difference = layer_module.gradient_against_difference()
    assert abs(slope - difference) <= 1e-2 * abs(difference)

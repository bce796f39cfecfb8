"""Sequence operators on the GPU against their 64-bit definitions (sequence_ref).

Tolerances: one rounding of the output type plus c roundings in 32 bits of the largest magnitude.  A norm's row sums
pass through at most 64 additions a lane and 8 between lanes, a gradient's dw through at most 64 rows a chain and 32
joins; a scan's state after t tokens has t roundings of its product, t of its sums, and the exponentials' (about 8
roundings each, the step size's among them), so c = 16 + 12 t, t at most the sequence's length; its gradients pass
through two such chains and a sum over tokens and channels."""
import random

import pytest
import torch

import sequence_ref as ref
from gpu_util import log
from sequence_ref import DT, close, leaf

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def iga():
    import implicit_gemm_amd
    return implicit_gemm_amd


def gen(seed):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g) * std).to(dtype)

    return rand


def strided(t, pad):
    """The same values as a part of wider rows."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), 7.0, dtype=t.dtype)
    wide[..., pad:] = t
    return wide.cuda()[..., pad:]


# ---------------------------------------------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (1, 257), (1100, 300), (1030, 1024), (2, 1537), (1025, 2048), (2, 4100), (3, 8192),
               (2, 16384), (0, 64), (1, 16383)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,C", NORM_SHAPES)
def test_norm_and_gradient(iga, rows, C, dtype):
    log("norm", rows, C, dtype)
    rand, dt = gen(rows * 31 + C), DT[dtype]
    x, res, dy, dh = (rand(rows, C, dtype=dt) for _ in range(4))
    w = rand(C)
    if rows > 1:
        x[1] = 0
        res[1] = 0                      # a row of zeros: r = eps^-1/2
    with_res = C % 2 == 0
    xd = strided(x, 3) if C < 5000 else x.cuda()
    y, h, r = iga.rms_norm(xd, w.cuda(), residual=res.cuda() if with_res else None, eps=1e-5)
    hr = ref.norm(x, res if with_res else None, w, 1e-5)[1]
    assert torch.equal(h.cpu(), hr)
    if not with_res:
        assert h is xd
    hl, wl = leaf(hr), leaf(w)
    yr, _, rr = ref.norm(hl, None, wl, 1e-5)
    close(y, yr, dt, 96, "y")
    close(r, rr, torch.float32, 96, "r", scale=rr.detach())
    for dhx in (None, dh):
        dx, dw = iga.rms_norm_grad(strided(dy, 5), h, w.cuda(), r, dh=dhx.cuda() if dhx is not None else None)
        dxr, dwr = ref.grads((yr,), (dy.double(),), (hl, wl)) if rows else (hl, torch.zeros(C))
        if dhx is not None:
            dxr = dxr + dhx.double()
        # the rows of zeros have r = 316, so each row is measured against its own largest terms
        top = ((dy.double() * w.double()).abs().amax(1, keepdim=True) * rr.detach()[:, None] * 2 + 4) if rows else None
        close(dx, dxr, dt, 160, "dx", scale=top)
        close(dw, dwr, torch.float32, 256 + rows, "dw")
        yr, _, rr = ref.norm(hl, None, wl, 1e-5)


def e4m3_expected(y, group):
    """Scales and the values q stands for, before their rounding."""
    M, C = y.shape
    g = group or C
    scale = torch.stack([p.abs().amax(1) / 448 for p in y.split(g, 1)], 1)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return scale, y / scale.repeat_interleave(g, 1)[:, :C]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,C,group", [(3, 300, 0), (2, 300, 32), (5, 300, 64), (1, 2048, 128), (1100, 520, 256),
                                          (1027, 1537, 128), (2, 7, 32), (1, 16384, 256), (2, 5000, 0), (0, 128, 128)])
def test_norm_e4m3(iga, rows, C, group, dtype):
    log("norm e4m3", rows, C, group, dtype)
    rand, dt = gen(rows + C + group), DT[dtype]
    x, res, w = rand(rows, C, dtype=dt), rand(rows, C, dtype=dt, std=2.0), rand(C)
    if rows > 1:
        x[1] = 0
        res[1] = 0
    q, scale, h = iga.rms_norm_e4m3(strided(x, 1), w.cuda(), residual=res.cuda(), group=group)
    y, hr, _ = ref.norm(x, res, w, 1e-5)
    assert torch.equal(h.cpu(), hr) and q.dtype == torch.float8_e4m3fn
    if rows == 0:
        assert q.shape == (0, C) and scale.shape == (0, -(-C // (group or C)))
        return
    sr, qr = e4m3_expected(y, group)
    close(scale, sr, torch.float32, 100, "scale", scale=sr)
    # half a step of e4m3: 2^-4 of the value, 2^-10 below the smallest normal number (2^-6); and the scale's error
    err = (q.cpu().double() - qr).abs()
    assert (err <= qr.abs() * (2.0 ** -4 + 200 * ref.EPS32) + 2.0 ** -10).all()
    assert q.cpu().float().abs().max() <= 448


def test_norm_keeps_nan_and_infinity_in_their_row(iga):
    x = torch.ones(3, 256)
    x[0, 5] = float("nan")
    x[1, 7] = float("inf")
    y, h, r = iga.rms_norm(x.cuda(), torch.ones(256).cuda())
    assert y[0].isnan().all() and y[1, 7].isnan() and bool((y[1, :7] == 0).all()) and bool(torch.isfinite(y[2]).all())
    q, scale, _ = iga.rms_norm_e4m3(x.cuda(), torch.ones(256).cuda(), group=128)
    assert scale[0].isnan().all() and scale[1, 0].isnan() and bool(torch.isfinite(scale[2]).all())


def test_norm_e4m3_below_the_normal_range(iga):
    """A scale below the normal range can be rounded to far less than max|y| / 448: the codes stay finite.  x = 1 and
    eps = 0 make y = w."""
    unit = 2.0 ** -149
    tops = torch.tensor([1, 223, 225, 313, 470, 667, 673, 6048, 100000, 2.0 ** 33])      # of the groups, in units
    w = (torch.linspace(-1, 1, 32)[None, :] * tops[:, None] * unit).double().flatten().float()
    for group, shape in ((32, (len(tops), 32)), (0, (1, -1))):
        q, scale, _ = iga.rms_norm_e4m3(torch.ones(2, len(w)).cuda(), w.cuda(), eps=0.0, group=group)
        want = w.view(shape).abs().amax(1) / 448           # 32 bits, denormals among them
        want = torch.where(want == 0, torch.ones_like(want), want)
        assert torch.equal(scale.cpu(), want.expand(2, -1))
        v = (w.view(shape).double() / want.double()[:, None]).clamp(-448, 448).flatten()
        got = q.cpu().float().double()
        assert bool(torch.isfinite(got).all()) and float(got.abs().max()) <= 448
        assert bool(((got - v).abs() <= v.abs() * 2.0 ** -4 + 2.0 ** -10).all())


def test_norm_of_higher_rank_and_its_refusals(iga):
    rand = gen(1)
    x = rand(2, 3, 5, 64).cuda()
    w = rand(64).cuda()
    y, _, r = iga.rms_norm(x, w)
    assert y.shape == x.shape and r.shape == (2, 3, 5)
    assert torch.equal(y.view(-1, 64), iga.rms_norm(x.view(-1, 64), w)[0])
    assert torch.equal(iga.rms_norm(x[0, 0, 0], w)[0], y[0, 0, 0])
    for bad in (lambda: iga.rms_norm(x.transpose(0, 1), w), lambda: iga.rms_norm(x.transpose(2, 3), w),
                lambda: iga.rms_norm(x, w.bfloat16()), lambda: iga.rms_norm(x, w[:32]),
                lambda: iga.rms_norm(x, w, residual=x[0]), lambda: iga.rms_norm(x.double(), w),
                lambda: iga.rms_norm_e4m3(x, w, group=100), lambda: iga.rms_norm(x, w.cpu()),
                lambda: iga.rms_norm_grad(x, x, w, r[0])):
        with pytest.raises((ValueError, TypeError, iga.ConvWgradError)):
            bad()


# --------------------------------------------------------------------------------------------------- convolution

PACKED = [[0, 1, 1, 3, 40, 41], [0, 0, 16, 48, 113], [0, 0], [0, 200]]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("W,D,act,offsets,tail", [
    (4, 64, True, None, 0), (2, 5, False, None, 0), (3, 130, True, None, 0), (4, 1, True, PACKED[0], 0),
    (4, 600, True, PACKED[0], 7), (3, 67, False, PACKED[1], 33), (2, 256, True, PACKED[2], 20), (4, 12, True, PACKED[3], 0),
    (4, 8, True, PACKED[2], 0)])
@pytest.mark.parametrize("carried", [False, True])
def test_conv_and_gradient(iga, W, D, act, offsets, tail, carried, dtype):
    log("conv", W, D, act, offsets, tail, carried, dtype)
    rand, dt = gen(W * 100 + D), DT[dtype]
    shape = (3, 37) if offsets is None else (offsets[-1] + tail,)
    S = 3 if offsets is None else len(offsets) - 1
    x, dy = rand(*shape, D, dtype=dt), rand(*shape, D, dtype=dt)
    w, b = rand(D, W, std=0.5), rand(D) if D != 5 else None
    P = S + 2
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(D))[:S].int()
    pool = rand(P, W - 1, D, dtype=dt)
    state = pool[slots.long()] if carried else None
    dlast = rand(S, W - 1, D, dtype=dt) if carried else None
    off = torch.tensor(offsets, dtype=torch.int32).cuda() if offsets is not None else None
    xd = strided(x, 3)
    kw = dict(silu=act, offsets=off)
    if carried:
        kw.update(state=pool.cuda(), slots=slots.cuda())
    out = torch.full((P, W - 1, D), 5.0, dtype=dt).cuda() if carried else None
    wd, bd = w.cuda(), b.cuda() if b is not None else None
    y, last = iga.causal_conv(xd, wd, bd, state_out=out, **kw)
    xl, wl, bl, sl = leaf(x), leaf(w), leaf(b), leaf(state)
    yr, lr = ref.conv(xl, wl, bl, act, offsets, sl)
    c = 16
    close(y, yr, dt, c, "y")
    if carried:
        want = torch.full((P, W - 1, D), 5.0, dtype=dt)
        want[slots.long()] = lr.detach().to(dt)
        assert torch.equal(last.cpu(), want)
        inplace = pool.cuda()
        y2, last2 = iga.causal_conv(xd, wd, bd, silu=act, offsets=off, state=inplace, slots=slots.cuda())
        assert last2 is inplace and torch.equal(y2, y)
        want = pool.clone()
        want[slots.long()] = lr.detach().to(dt)
        assert torch.equal(inplace.cpu(), want)
    else:
        assert torch.equal(last.cpu(), lr.detach().to(dt))
    got = iga.causal_conv_grad(strided(dy, 1), xd, wd, bd, dstate_out=dlast.cuda() if carried else None, **kw)
    inside = dy.double()
    if tail:
        inside[offsets[-1]:] = 0
    exp = ref.grads((yr, lr), (inside, dlast.double() if carried else None), (xl, wl, bl, sl))
    n = x.numel() // D
    close(got[0], exp[0], dt, 64, "dx")
    close(got[1], exp[1], torch.float32, 64 + n, "dw")
    if b is not None:
        close(got[2], exp[2], torch.float32, 64 + n, "db")
    else:
        assert got[2] is None
    if carried:
        close(got[3], exp[3], dt, 64, "dstate")
    else:
        assert got[3] is None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("W,D,act,offsets,tail", [
    (4, 256, True, None, 0), (3, 512, False, None, 0), (2, 256, True, [0, 70, 70, 71, 180, 183], 9),
    (4, 512, True, [0, 70, 70, 71, 180, 183], 9), (4, 128, True, [0, 33, 66, 67, 200], 0), (3, 256, True, [0, 1, 3, 130], 40)])
@pytest.mark.parametrize("carried", [False, True])
def test_conv_of_whole_channel_blocks(iga, W, D, act, offsets, tail, carried, dtype):
    """The kernels without channel checks (blocks of 256 channels forward, 128 backward), over sequences of several pieces,
    of one, and of none."""
    test_conv_and_gradient(iga, W, D, act, offsets, tail, carried, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_conv_long_has_many_pieces_a_workgroup(iga, dtype):
    """More pieces than partial sums: each workgroup of the gradient walks along several."""
    rand, dt = gen(3), DT[dtype]
    x, dy, w, b = rand(2, 20000, 8, dtype=dt), rand(2, 20000, 8, dtype=dt), rand(8, 4, std=0.5), rand(8)
    y, _ = iga.causal_conv(x.cuda(), w.cuda(), b.cuda(), silu=True)
    dx, dw, db, _ = iga.causal_conv_grad(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), silu=True)
    xl, wl, bl = leaf(x), leaf(w), leaf(b)
    yr, _ = ref.conv(xl, wl, bl, True, None, None)
    exp = ref.grads((yr,), (dy.double(),), (xl, wl, bl))
    close(y, yr, dt, 16, "y")
    close(dx, exp[0], dt, 64, "dx")
    close(dw, exp[1], torch.float32, 2000, "dw")
    close(db, exp[2], torch.float32, 2000, "db")


@pytest.mark.parametrize("dtype", TYPES)
def test_conv_of_long_pieces(iga, dtype):
    """Enough tokens for pieces of 64, whose windows and gradients pass many batches; odd lengths end inside one."""
    rand, dt = gen(4), DT[dtype]
    S, L, D = 3, 90001, 8
    x, dy, w, b = rand(S, L, D, dtype=dt), rand(S, L, D, dtype=dt), rand(D, 4, std=0.5), rand(D)
    y, _ = iga.causal_conv(x.cuda(), w.cuda(), b.cuda(), silu=True)
    dx, dw, db, _ = iga.causal_conv_grad(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), silu=True)
    xl, wl, bl = leaf(x), leaf(w), leaf(b)
    yr, _ = ref.conv(xl, wl, bl, True, None, None)
    exp = ref.grads((yr,), (dy.double(),), (xl, wl, bl))
    close(y, yr, dt, 16, "y")
    close(dx, exp[0], dt, 64, "dx")
    close(dw, exp[1], torch.float32, 64 + S * L, "dw")
    close(db, exp[2], torch.float32, 64 + S * L, "db")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [128, 70])
def test_conv_gradient_of_an_empty_sequence_ignores_its_window(iga, D, dtype):
    rand, dt = gen(D), DT[dtype]
    off = torch.tensor([0, 20, 20, 20, 53, 53], dtype=torch.int32).cuda()
    x, dy, w, b = rand(53, D, dtype=dt).cuda(), rand(53, D, dtype=dt).cuda(), rand(D, 4, std=0.5).cuda(), rand(D).cuda()
    state, dlast = rand(5, 3, D, dtype=dt).cuda(), rand(5, 3, D, dtype=dt).cuda()
    state[[1, 2, 4]] = 0
    kw = dict(silu=True, offsets=off, dstate_out=dlast)
    want = iga.causal_conv_grad(dy, x, w, b, state=state, **kw)
    state[1], state[2, 1], state[4] = float("nan"), float("inf"), -float("inf")
    got = iga.causal_conv_grad(dy, x, w, b, state=state, **kw)
    for g, e in zip(got, want):
        assert bool(torch.isfinite(g).all()) and torch.equal(g, e)
    assert torch.equal(got[3][[1, 2, 4]], dlast[[1, 2, 4]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("keep", ["state_out", "copy", "copy in order"])
def test_conv_gradient_beside_a_pool(iga, keep, dtype):
    """The gradient reads the windows before the sequences, which a call with slots writes over: the ways of keeping them
    that the two calls name, against the definition."""
    rand, dt = gen(15), DT[dtype]
    offsets, P, D, W = [0, 1, 8, 8, 60], 6, 70, 4
    x, dy, w, b = rand(60, D, dtype=dt), rand(60, D, dtype=dt), rand(D, W, std=0.5), rand(D)
    pool, slots = rand(P, W - 1, D, dtype=dt), torch.tensor([4, 0, 5, 2], dtype=torch.int32)
    state, kw = pool.cuda(), dict(silu=True, offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
    xd, wd, bd, at = x.cuda(), w.cuda(), b.cuda(), slots.cuda()
    if keep == "state_out":
        iga.causal_conv(xd, wd, bd, slots=at, state=state, state_out=torch.empty_like(state), **kw)
        got = iga.causal_conv_grad(dy.cuda(), xd, wd, bd, slots=at, state=state, **kw)
    else:
        before = state.clone() if keep == "copy" else state[at.long()]
        _, new = iga.causal_conv(xd, wd, bd, slots=at, state=state, **kw)
        assert new is state and not torch.equal(state, pool.cuda())
        got = iga.causal_conv_grad(dy.cuda(), xd, wd, bd, state=before, slots=at if keep == "copy" else None, **kw)
    leaves = [leaf(x), leaf(w), leaf(b), leaf(pool[slots.long()])]
    yr, _ = ref.conv(*leaves[:3], True, offsets, leaves[3])
    for name, g, e, t, c in zip(("dx", "dw", "db", "dstate"), got, ref.grads((yr,), (dy.double(),), leaves),
                                (dt, torch.float32, torch.float32, dt), (64, 64 + 60, 64 + 60, 64)):
        close(g, e, t, c, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("W,D,S", [(4, 300, 1), (4, 1030, 5), (2, 3, 4), (3, 64, 2)])
def test_conv_step_matches_prompt(iga, W, D, S, dtype):
    """Tokens one at a time give the prompt's outputs bit for bit (the same sums in the same order) and its window."""
    rand, dt = gen(D), DT[dtype]
    T = 6
    x, w, b = strided(rand(S, T, D, dtype=dt), 2), rand(D, W, std=0.5).cuda(), rand(D).cuda()
    pool = rand(S + 1, W - 1, D, dtype=dt).cuda()
    slots = torch.arange(S, 0, -1, dtype=torch.int32).cuda()
    whole = pool.clone()
    y, _ = iga.causal_conv(x, w, b, silu=True, state=whole, slots=slots)
    steps = [iga.causal_conv_step(x[:, t], pool, w, b, silu=True, slots=slots) for t in range(T)]
    assert torch.equal(torch.stack(steps, 1), y) and torch.equal(pool, whole)


def test_slots_outside_the_pool_have_no_state(iga):
    rand = gen(9)
    pool, w, x = rand(4, 3, 64).cuda(), rand(64, 4).cuda(), rand(3, 64).cuda()
    slots = torch.tensor([-1, 2, 4], dtype=torch.int32).cuda()
    before = pool.clone()
    y = iga.causal_conv_step(x, pool, w, slots=slots)
    assert torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]])
    assert torch.equal(pool[2], torch.cat([before[2, 1:], x[1:2]]))
    zero = iga.causal_conv_step(x, torch.zeros(3, 3, 64).cuda(), w)
    assert torch.equal(y[[0, 2]], zero[[0, 2]])
    A, Bc = -torch.rand(64, 16).cuda() - 0.1, rand(3, 1, 16).cuda()
    states = rand(4, 64, 16).cuda()
    before = states.clone()
    y = iga.selective_scan_step(x, x, A, Bc, Bc, states, softplus=True, slots=slots)
    assert torch.equal(states[[0, 1, 3]], before[[0, 1, 3]]) and not torch.equal(states[2], before[2])
    zero = iga.selective_scan_step(x, x, A, Bc, Bc, torch.zeros(3, 64, 16).cuda(), softplus=True)
    assert torch.equal(y[[0, 2]], zero[[0, 2]])
    y2, _, _ = iga.selective_scan(x, x, A, Bc, Bc, softplus=True, state=before.clone(), slots=slots,
                                  offsets=torch.arange(4, dtype=torch.int32).cuda())
    close(y2, y.double(), torch.float32, 64, "prompt of one token")


# ---------------------------------------------------------------------------------------------------------- scan

def scan_case(D, N, G, offsets, tail, dtype, opts, seed, L=37, S=2):
    rand, dt = gen(seed), DT[dtype]
    shape = (S, L) if offsets is None else (offsets[-1] + tail,)
    S = S if offsets is None else len(offsets) - 1
    case = dict(u=rand(*shape, D, dtype=dt), delta=rand(*shape, D, std=0.5, dtype=dt),
                A=-(torch.arange(1, N + 1).float() * (0.8 + 0.4 * torch.rand(D, N, generator=torch.Generator().manual_seed(seed)))),
                B=rand(*shape, G, N, dtype=dt), C=rand(*shape, G, N, dtype=dt),
                skip=rand(D) if "skip" in opts else None, z=rand(*shape, D, dtype=dt) if "z" in opts else None,
                bias=rand(D) - 2 if "bias" in opts else None, softplus="softplus" in opts,
                state=rand(S, D, N) if "state" in opts else None, dy=rand(*shape, D, dtype=dt),
                dlast=rand(S, D, N) if "last" in opts else None, offsets=offsets, S=S, dt=dt)
    if not case["softplus"]:
        case["delta"] = (case["delta"].float().abs() * 0.2 + 0.01).to(dt)
        if case["bias"] is not None:
            case["bias"] = case["bias"].abs() * 0.05
    return case


def run_scan(iga, c, max_len=None, grad=True, stream=None):
    def dev(t):
        return t.cuda() if t is not None else None

    off = torch.tensor(c["offsets"], dtype=torch.int32).cuda() if c["offsets"] is not None else None
    A = c["A"].cuda()
    kw = dict(skip=dev(c["skip"]), z=strided(c["z"], 4) if c["z"] is not None else None, delta_bias=dev(c["bias"]),
              softplus=c["softplus"], offsets=off, max_len=max_len, state=dev(c["state"]), stream=stream)
    B, C = strided(c["B"], 5), strided(c["C"], 3)
    u, delta = c["u"].cuda(), strided(c["delta"], 1)
    y, last, saved = iga.selective_scan(u, delta, A, B, C, save=grad, **kw)
    if not grad:
        return y, last
    return y, last, iga.selective_scan_grad(strided(c["dy"], 2), u, delta, A, B, C, saved, dstate_out=dev(c["dlast"]), **kw)


ALL = ("skip", "z", "bias", "softplus", "state", "last")
SCAN = [
    # D, N, G, offsets, tail, options, L
    (64, 16, 1, None, 0, ALL, 37), (1, 1, 1, None, 0, (), 1), (37, 11, 1, None, 0, ALL, 17), (130, 32, 1, None, 0, ALL, 16),
    (66, 8, 2, None, 0, ("softplus", "state"), 65), (200, 24, 2, None, 0, ("z", "bias", "softplus", "last"), 33),
    (70, 4, 1, None, 0, ("skip",), 15), (64, 16, 1, None, 0, ALL, 0), (96, 16, 1, None, 0, ALL, 150), (33, 20, 3, None, 0, ALL, 130),
    (64, 16, 1, PACKED[0], 0, ALL, 0), (65, 9, 1, PACKED[1], 33, ALL, 0), (8, 16, 2, PACKED[2], 20, ALL, 0),
    (48, 16, 1, PACKED[3], 0, ("softplus",), 0), (40, 8, 1, PACKED[1], 1, ("z", "state"), 0), (64, 16, 1, PACKED[2], 0, ALL, 0),
    (24, 3, 1, None, 0, ("z", "softplus", "bias"), 64),
]


def check_scan(c, got, L):
    y, last, g = got if len(got) == 3 else (*got, None)
    names = ("u", "delta", "A", "B", "C", "skip", "z", "bias", "state")
    leaves = [leaf(c[n]) for n in names]
    yr, hr = ref.scan(*leaves[:5], leaves[5], leaves[6], leaves[7], c["softplus"], c["offsets"], leaves[8])
    cc = 16 + 12 * L
    dt = c["dt"]
    close(y, yr, dt, cc, "y")
    close(last, hr, torch.float32, cc, "state")
    if g is None:
        return
    inside = c["dy"].double()
    if c["offsets"] is not None:
        inside[c["offsets"][-1]:] = 0
    exp = ref.grads((yr, hr), (inside, c["dlast"].double() if c["dlast"] is not None else None), leaves)
    rows = c["u"].numel() // c["u"].shape[-1]
    for name, e, t, extra in zip(("du", "ddelta", "dA", "dB", "dC", "dskip", "dz", "ddelta_bias", "dstate"), exp,
                                 (dt, dt, torch.float32, dt, dt, torch.float32, dt, torch.float32, torch.float32),
                                 (0, 0, rows, 64, 64, rows, 0, rows, 0)):
        if e is None:
            assert getattr(g, name) is None, name
        else:
            close(getattr(g, name), e, t, 4 * cc + extra, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,N,G,offsets,tail,opts,L", SCAN)
def test_scan_and_gradient(iga, D, N, G, offsets, tail, opts, L, dtype):
    log("scan", D, N, G, offsets, tail, opts, L, dtype)
    c = scan_case(D, N, G, offsets, tail, dtype, opts, D + N + L, L=L)
    longest = L if offsets is None else max(b - a for a, b in zip(offsets, offsets[1:]))
    check_scan(c, run_scan(iga, c), longest)
    if offsets is not None:
        # told the longest length: the short ones go in one launch, with the same results to rounding
        check_scan(c, run_scan(iga, c, max_len=max(longest, 1)), longest)
        y, _ = run_scan(iga, c, max_len=1, grad=False)      # a hint that is wrong changes nothing either
        check_scan(c, (y, run_scan(iga, c, grad=False)[1]), longest)


# Long scans: a state forgets, so that its error comes from the tokens within its memory, 1 / (1 - e^(D A)) of the slowest
# state: that many roundings, where they are fewer than the tokens.  Without softplus D is 0.01 and more, which makes it 125
# at most, with a good part of every state handed from piece to piece.
SLOW = ("skip", "z", "bias", "state", "last")


def memory(c):
    dt = c["delta"].double() + (c["bias"].double() if c["bias"] is not None else 0)
    dt = torch.logaddexp(dt, torch.zeros_like(dt)) if c["softplus"] else dt
    slow = (dt.amin(tuple(range(dt.dim() - 1)))[:, None] * -c["A"].double()).min()
    return round(float(1 / -torch.expm1(-slow)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,N,G,S,L,opts", [
    (24, 11, 1, 2, 1100, SLOW), (64, 16, 1, 1, 1030, SLOW),          # 69 and 65 pieces: the join takes another round
    (64, 8, 1, 2, 300, SLOW), (128, 32, 1, 2, 150, SLOW), (128, 32, 2, 1, 100, ALL),   # whole blocks of channels and states
    (64, 4, 64, 2, 1100, SLOW)])                                     # pieces of 64 tokens
def test_long_scan_and_gradient(iga, D, N, G, S, L, opts, dtype):
    log("long scan", D, N, G, S, L, dtype)
    c = scan_case(D, N, G, None, 0, dtype, opts, D + N, L=L, S=S)
    check_scan(c, run_scan(iga, c), min(L, memory(c)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_scan_and_gradient(iga, dtype):
    """Pieces of 64 tokens, four tiles of the gradient, in whole blocks of channels."""
    c = scan_case(4096, 8, 64, None, 0, dtype, SLOW, 5, L=1100, S=2)
    check_scan(c, run_scan(iga, c), min(1100, memory(c)))


@pytest.mark.parametrize("max_len", [None, 500, 1, 65])
@pytest.mark.parametrize("dtype", TYPES)
def test_packed_scan_by_the_join_of_one_wave(iga, dtype, max_len):
    """50 sequences x 3 channel blocks x 16 states are joined by a wave each, 32 pieces of the longest in two rounds, where
    no sequence is known to be longer (500; 65, which is wrong, as is 1, with which none is split); else by four."""
    offsets = [0]
    for i in range(50):
        offsets.append(offsets[-1] + {3: 500, 20: 257, 21: 256, 40: 273}.get(i, [0, 1, 15, 16, 17, 40][i % 6]))
    c = scan_case(192, 16, 1, offsets, 11, dtype, SLOW, 6)
    check_scan(c, run_scan(iga, c, max_len=max_len), min(500, memory(c)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("max_len", [1, 65])
def test_scan_with_a_wrong_longest_length(iga, dtype, max_len):
    """Outputs, states and gradients do not depend on max_len being right, in one piece (1) and split (65)."""
    c = scan_case(40, 11, 2, [0, 300, 300, 301, 520], 7, dtype, SLOW, 7)
    check_scan(c, run_scan(iga, c, max_len=max_len), min(300, memory(c)))


@pytest.mark.parametrize("dtype", TYPES)
def test_scan_of_many_short_sequences(iga, dtype):
    rng = random.Random(3)
    offsets = [0]
    for _ in range(150):
        offsets.append(offsets[-1] + rng.choice([0, 1, 1, 2, 3, 9]))
    c = scan_case(24, 16, 1, offsets, 5, dtype, ALL, 77)
    check_scan(c, run_scan(iga, c), 9)
    check_scan(c, run_scan(iga, c, max_len=9), 9)


@pytest.mark.parametrize("dtype", TYPES)
def test_scan_with_more_pieces_than_workgroups(iga, dtype):
    """A narrow layer over many sequences: the gradient's workgroups walk along several pieces each."""
    c = scan_case(3, 2, 1, None, 0, dtype, ALL, 78, L=18, S=4500)
    check_scan(c, run_scan(iga, c), 18)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,N,G,S", [(64, 16, 1, 3), (37, 11, 1, 1), (66, 32, 2, 5), (300, 8, 3, 2), (5, 1, 1, 2)])
def test_scan_step_matches_prompt(iga, D, N, G, S, dtype):
    T = 5
    c = scan_case(D, N, G, None, 0, dtype, ALL, D, L=T, S=S)
    y, last, _ = run_scan(iga, c)
    pool = torch.zeros(S + 2, D, N).cuda()
    slots = torch.arange(S + 1, 1, -1, dtype=torch.int32).cuda()
    pool[slots.long()] = c["state"].cuda()
    u, delta, z, B, C = (strided(c[k], 4) for k in ("u", "delta", "z", "B", "C"))
    args = dict(skip=c["skip"].cuda(), delta_bias=c["bias"].cuda(), softplus=True, slots=slots)
    outs = [iga.selective_scan_step(u[:, t], delta[:, t], c["A"].cuda(), B[:, t], C[:, t], pool, z=z[:, t], **args)
            for t in range(T)]
    check_scan(c, (torch.stack(outs, 1), pool[slots.long()]), T)
    assert bool((pool[:2] == 0).all())
    other = torch.full_like(pool, 3.0)
    iga.selective_scan_step(u[:, 0], delta[:, 0], c["A"].cuda(), B[:, 0], C[:, 0], pool, z=z[:, 0], state_out=other, **args)
    assert bool((other[:2] == 3).all())


@pytest.mark.slow
def test_scan_of_very_many_sequences(iga):
    """2^14 sequences of 4096 channels x 16 states (a join of them would not fit a launch): a token of each, and packed
    prompts of 0 .. 3 tokens, give what the two halves give, bit for bit."""
    S, D, N = 1 << 14, 4096, 16
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    A, bias = -torch.rand(D, N, device="cuda") - 0.1, torch.full((D,), -1.0, device="cuda")
    kw = dict(delta_bias=bias, softplus=True)
    state = torch.randn(S, D, N, generator=g, device="cuda")
    halves = (slice(0, S // 2), slice(S // 2, S))
    u, B = rand(S, D), rand(S, 1, N)
    new = torch.empty_like(state)
    y = iga.selective_scan_step(u, u, A, B, B, state, state_out=new, **kw)
    for h in halves:
        part = torch.empty_like(state[h])
        assert torch.equal(y[h], iga.selective_scan_step(u[h], u[h], A, B[h], B[h], state[h], state_out=part, **kw))
        assert torch.equal(new[h], part)
    lens = torch.arange(S, device="cuda") % 4
    off = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    cut = int(off[S // 2])
    u, B = rand(int(off[-1]), D), rand(int(off[-1]), 1, N)
    y = iga.selective_scan(u, u, A, B, B, offsets=off, state=state, state_out=new, **kw)[0]
    for h, r, o in ((halves[0], slice(0, cut), off[:S // 2 + 1]), (halves[1], slice(cut, None), off[S // 2:] - cut)):
        part = torch.empty_like(state[h])
        y2 = iga.selective_scan(u[r], u[r], A, B[r], B[r], offsets=o.int(), max_len=3, state=state[h], state_out=part, **kw)[0]
        assert torch.equal(y[r], y2) and torch.equal(new[h], part)


@pytest.mark.parametrize("split", [False, True])
def test_scan_in_place_and_in_two_halves(iga, split):
    """A prompt in two calls, its state carried in place, gives the states of one call; sums are split elsewhere, so
    equal to rounding."""
    L = 160 if split else 40
    c = scan_case(50, 16, 1, None, 0, "f32", ALL, 21, L=L)
    y, last = run_scan(iga, c, grad=False)
    state = c["state"].cuda()
    k = L // 2 + 3
    kw = dict(skip=c["skip"].cuda(), delta_bias=c["bias"].cuda(), softplus=True, state=state, state_out=state)
    parts = []
    for lo, hi in ((0, k), (k, L)):
        u, d, z, B, C = (c[n].cuda()[:, lo:hi] for n in ("u", "delta", "z", "B", "C"))
        parts.append(iga.selective_scan(u, d, c["A"].cuda(), B, C, z=z, **kw)[0])
    close(torch.cat(parts, 1), y.double(), torch.float32, 16 + 12 * L, "y")
    close(state, last.double(), torch.float32, 16 + 12 * L, "state")


@pytest.mark.parametrize("late", [True, False])
def test_scan_of_growing_states(iga, late):
    """Where A D is positive a state of zero stays zero and a tiny one grows to what it should, though e^(A sum D) of the
    tokens between overflows (late: inputs in the last 20 tokens and gradients in the first 10, so that both directions
    carry zeros; else a tiny first state)."""
    c = scan_case(24, 3, 1, None, 0, "f32", ("skip", "state", "last"), 31, L=400 if late else 100)
    c["A"] = c["A"].abs()                      # 0.8 .. 3.6
    c["delta"] = torch.full_like(c["delta"], 0.4 if late else 0.28)
    if late:
        c["u"][:, :380], c["dy"][:, 10:] = 0, 0
        c["state"], c["dlast"] = torch.zeros_like(c["state"]), torch.zeros_like(c["dlast"])
        check_scan(c, run_scan(iga, c), 400)
    else:
        c["u"] = torch.zeros_like(c["u"])
        c["state"] *= 1e-30
        check_scan(c, run_scan(iga, c, grad=False), 100)


@pytest.mark.parametrize("L", [37, 64, 100])
def test_scan_of_infinite_inputs_and_decays(iga, L):
    """A of -inf forgets at each token; an infinite last input gives an infinite state, whatever the length is a multiple
    of."""
    c = scan_case(24, 8, 1, None, 0, "f32", ("skip", "state"), 32, L=L)
    c["B"], c["C"], c["skip"] = c["B"].abs() + 0.1, c["C"].abs() + 0.1, c["skip"].abs()
    c["A"][:, 2] = -float("inf")
    y, last = run_scan(iga, c, grad=False)
    assert bool(torch.isfinite(last).all()) and bool(torch.isfinite(y).all())
    check_scan(c, (y, last), L)
    c["u"][0, -1, 3], c["u"][1, -1, 4] = float("inf"), -float("inf")
    y, last = run_scan(iga, c, grad=False)
    check_scan(c, (y, last), L)
    assert bool((last[0, 3] == float("inf")).all()) and bool((last[1, 4] == -float("inf")).all())
    state = c["state"].cuda()
    out = iga.selective_scan_step(c["u"].cuda()[:, 0], c["delta"].cuda()[:, 0], c["A"].cuda(), c["B"].cuda()[:, 0],
                                  c["C"].cuda()[:, 0], state, skip=c["skip"].cuda())
    one = {k: v[:, :1] if k in ("u", "delta", "B", "C", "dy") else v for k, v in c.items()}
    check_scan(one, (out[:, None], state), 1)


@pytest.mark.parametrize("L", [37, 64, 100])
def test_scan_gradient_of_an_infinite_last_gradient(iga, L):
    c = scan_case(24, 8, 1, None, 0, "f32", ("skip",), 33, L=L)
    for k in ("B", "C", "skip"):
        c[k] = c[k].abs() + 0.1
    c["dy"][0, -1, 3], c["dy"][1, -1, 4] = float("inf"), -float("inf")
    du = run_scan(iga, c)[2].du
    leaves = [leaf(c[n]) for n in ("u", "delta", "A", "B", "C", "skip")]
    y, _ = ref.scan(*leaves, None, None, False, None, None)
    want = ref.grads((y,), (c["dy"].double(),), leaves)[0]
    assert bool((want[0, :, 3] == float("inf")).all()) and bool((want[1, :, 4] == -float("inf")).all())
    close(du, want, torch.float32, 4 * (16 + 12 * L), "du")


def test_scan_gradient_against_differences(iga):
    """The directional derivative from the GPU's gradients against central differences of the 64-bit definition."""
    c = scan_case(20, 16, 1, None, 0, "f32", ALL, 8, L=70)
    _, _, g = run_scan(iga, c)
    names = ("u", "delta", "A", "B", "C", "skip", "z", "bias", "state")
    got = (g.du, g.ddelta, g.dA, g.dB, g.dC, g.dskip, g.dz, g.ddelta_bias, g.dstate)
    ins = [c[n].double() for n in names]
    direction = [torch.randn(t.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i)) for i, t in enumerate(ins)]

    def loss(e):
        v = [t + e * d for t, d in zip(ins, direction)]
        y, h = ref.scan(*v[:5], v[5], v[6], v[7], True, None, v[8])
        return (y * c["dy"].double()).sum() + (h * c["dlast"].double()).sum()

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [(a.double().cpu() * d) for a, d in zip(got, direction)]
    have, mass = sum(t.sum() for t in terms), sum(t.abs().sum() for t in terms)
    assert abs(have - want) <= (4 * (16 + 12 * 70) * ref.EPS32) * mass + 1e-6 * abs(want)


def test_results_do_not_change_from_run_to_run(iga):
    c = scan_case(130, 16, 1, None, 0, "bf16", ALL, 4, L=300)
    first, second = run_scan(iga, c), run_scan(iga, c)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    assert all(torch.equal(a, b) for a, b in zip(first[2], second[2]))


def test_scan_refusals(iga):
    rand = gen(2)
    u, A, B = rand(2, 5, 8).cuda(), -torch.ones(8, 4).cuda(), rand(2, 5, 1, 4).cuda()
    off = torch.tensor([0, 5], dtype=torch.int32).cuda()
    y, last, saved = iga.selective_scan(u, u, A, B, B, save=True)
    for bad in (lambda: iga.selective_scan(u, u[:1], A, B, B), lambda: iga.selective_scan(u, u, A.half(), B, B),
                lambda: iga.selective_scan(u, u, A, B, B.half()), lambda: iga.selective_scan(u, u, A[:4], B, B),
                lambda: iga.selective_scan(u, u, A, B[:, :, :, :3], B), lambda: iga.selective_scan(u, u, A, B, B, offsets=off),
                lambda: iga.selective_scan(u[0], u[0], A, B[0], B[0], offsets=off.long()),
                lambda: iga.selective_scan(u, u, A, B, B, state=last[:1]),
                lambda: iga.selective_scan(u, u, A, B, B, state=last.half()),
                lambda: iga.selective_scan(u, u, A, B, B, skip=torch.ones(7).cuda()),
                lambda: iga.selective_scan(u.transpose(1, 2), u, A, B, B),
                lambda: iga.selective_scan(u, u, -torch.ones(8, 40).cuda(), rand(2, 5, 1, 40).cuda(), rand(2, 5, 1, 40).cuda()),
                lambda: iga.selective_scan_step(u, u, A, B, B, last),
                lambda: iga.selective_scan_grad(u, u, u, A, B, B, saved[:-1]),
                lambda: iga.causal_conv(u, rand(8, 5).cuda()), lambda: iga.causal_conv(u, rand(7, 4).cuda()),
                lambda: iga.causal_conv(u, rand(8, 4).cuda(), state=u)):
        with pytest.raises((ValueError, TypeError, iga.ConvWgradError)):
            bad()


def test_conv_refuses_its_filters_before_it_allocates(iga):
    x = torch.zeros(1, 2, 1 << 15).cuda()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for w in (torch.zeros(1 << 15).cuda(), torch.tensor(1.0).cuda(), torch.zeros(4, 1 << 15).cuda(), torch.zeros(1 << 15, 0).cuda()):
        with pytest.raises(ValueError):
            iga.causal_conv(x, w)
    assert torch.cuda.max_memory_allocated() <= before + (1 << 20)


# ------------------------------------------------------------------------------------------------ streams, graphs

def test_on_another_stream(iga):
    c = scan_case(64, 16, 1, None, 0, "bf16", ALL, 6, L=200)
    want = run_scan(iga, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_scan(iga, c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[2], want[2]))
    x, w = torch.randn(4, 256).cuda(), torch.ones(256).cuda()
    side.wait_stream(torch.cuda.current_stream())
    y = iga.rms_norm(x, w, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, iga.rms_norm(x, w)[0])


def test_captured_into_a_graph(iga):
    """Norm, convolution and scan with their gradients in one graph: every replay, on new inputs and with eager work
    in between, gives the eager results."""
    rand = gen(12)
    S, L, D, N = 2, 130, 64, 16
    x, dy = rand(S, L, D).cuda(), rand(S, L, D).cuda()
    w, cw, cb = rand(D).cuda(), rand(D, 4).cuda(), rand(D).cuda()
    A, bias = -torch.rand(D, N).cuda() - 0.2, rand(D).cuda()
    B = rand(S, L, 1, N).cuda()
    pool, states = rand(S, 3, D).cuda(), rand(S, D, N).cuda()

    def work(pool, states):
        y, h, r = iga.rms_norm(x, w)
        v, _ = iga.causal_conv(y, cw, cb, silu=True)
        o, last, saved = iga.selective_scan(v, y, A, B, B, z=x, delta_bias=bias, softplus=True, save=True)
        g = iga.selective_scan_grad(dy, v, y, A, B, B, saved, z=x, delta_bias=bias, softplus=True)
        dv = iga.causal_conv_grad(g.du, y, cw, cb, silu=True)
        dx, dw = iga.rms_norm_grad(dv[0], h, w, r)
        t = iga.causal_conv_step(x[:, 0], pool, cw, cb, silu=True)
        t = iga.selective_scan_step(t, x[:, 1], A, B[:, 0], B[:, 1], states, delta_bias=bias, softplus=True)
        return [o, last, dx, dw, dv[1], g.dA, g.dB, t]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(pool.clone(), states.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(pool, states)
    for i in range(4):
        x.copy_(torch.randn(S, L, D, generator=torch.Generator().manual_seed(i)))
        p, s = pool.clone(), states.clone()
        want = work(p, s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert torch.equal(pool, p) and torch.equal(states, s)


# -------------------------------------------------------------------------------------------------- the whole layer

@pytest.fixture(scope="module")
def layer_module():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_layer.py")
    spec = importlib.util.spec_from_file_location("selective_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_by_tokens_matches_prompts(layer_module, dtype):
    """Four roundings to the element type lie between the layer's input and its output, on both sides, and the matrix
    products between them sum in other orders: sixteen half steps of the largest output cover them."""
    layer = layer_module.Layer(96, dtype=DT[dtype], seed=3)
    off = layer_module.steps_against_prompt(layer, [130, 5, 33, 17])
    assert off <= max(16 * ref.half_step(DT[dtype]), 1e-5)


def test_layer_gradient_against_difference(layer_module):
    """Central differences of a float32 loss: the step's square and the losses' rounding (2^-24 of their terms over the
    step) leave about a thousandth."""
    slope, difference = layer_module.gradient_against_difference()
    assert abs(slope - difference) <= 1e-2 * abs(difference)


# ------------------------------------------------------------------------------------------------ past 32-bit offsets

@pytest.mark.slow
def test_tensors_past_four_gigabytes(iga):
    """Rows whose byte offsets (and element offsets) pass 2^32: the end of a long sequence against the same tokens alone,
    from the carried window and state."""
    T, D, N, tail = 540_000, 4096, 4, 96
    g = torch.Generator(device="cuda").manual_seed(1)

    def big():
        return torch.randn(1, T, D, generator=g, device="cuda", dtype=torch.bfloat16)

    x, w, b = big(), torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    assert x.numel() > 1 << 31 and x.numel() * 2 > 1 << 32
    end = slice(T - tail, T)
    y, h, r = iga.rms_norm(x, torch.ones(D, device="cuda"), residual=x)
    y2, h2, r2 = iga.rms_norm(x[:, end], torch.ones(D, device="cuda"), residual=x[:, end])
    assert torch.equal(y[:, end], y2) and torch.equal(h[:, end], h2)
    dx, _ = iga.rms_norm_grad(y, h, torch.ones(D, device="cuda"), r)
    dx2, _ = iga.rms_norm_grad(y2, h2, torch.ones(D, device="cuda"), r2)
    assert torch.equal(dx[:, end], dx2)
    del y, h, dx
    log("past 4 GiB: norm done")
    window = x[:, T - tail - 3:T - tail].contiguous()
    u, last = iga.causal_conv(x, w, b, silu=True)
    u2, last2 = iga.causal_conv(x[:, end], w, b, silu=True, state=window)
    assert torch.equal(u[:, end], u2) and torch.equal(last, last2)
    dx = iga.causal_conv_grad(x, x, w, b, silu=True)[0]
    dx2 = iga.causal_conv_grad(x[:, end], x[:, end], w, b, silu=True, state=window)[0]
    assert torch.equal(dx[:, end], dx2)
    del dx, u
    log("past 4 GiB: convolution done")
    A = -torch.arange(1, N + 1, device="cuda").float().repeat(D, 1)
    B = torch.randn(1, T, 1, N, generator=g, device="cuda", dtype=torch.bfloat16)
    bias = torch.full((D,), -3.0, device="cuda")
    kw = dict(delta_bias=bias, softplus=True)
    y, last, saved = iga.selective_scan(x, x, A, B, B, save=True, **kw)
    _, before, _ = iga.selective_scan(x[:, :T - tail], x[:, :T - tail], A, B[:, :T - tail], B[:, :T - tail], **kw)
    y2, last2, saved2 = iga.selective_scan(x[:, end], x[:, end], A, B[:, end], B[:, end], state=before, save=True, **kw)
    close(y[:, end], y2.double(), torch.bfloat16, 16 + 12 * tail, "y")     # two roundings of one value: within two half steps
    close(last, last2.double(), torch.float32, 16 + 12 * tail, "state")
    del y
    full = iga.selective_scan_grad(x, x, x, A, B, B, saved, **kw)
    part = iga.selective_scan_grad(x[:, end], x[:, end], x[:, end], A, B[:, end], B[:, end], saved2, state=before, **kw)
    for name in ("du", "ddelta", "dB", "dC"):
        a, b2 = getattr(full, name)[:, end].double(), getattr(part, name).double()
        assert (a - b2).abs().max() <= 2.0 ** -7 * b2.abs().max(), name   # both rounded to bf16: at most one step apart
    log("past 4 GiB: scan done")

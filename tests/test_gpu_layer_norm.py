"""Layer norm and its gradient on the GPU against the definition in 64 bits.

Tolerances: one rounding of the output type plus roundings in 32 bits.  A row's sums pass through at most 64 additions a
lane and 8 between lanes, so m is off by at most 72 eps of the row's largest |h| and n = (h - m) r by that times r, plus
some 40 roundings of n itself (the sum of squares, its root, the products).  dx adds two such sums of dy w and dy w n.
dw's and db's terms pass through at most `rows` additions and 32 joins."""
import pytest
import torch

import sequence_ref as ref
from gpu_util import log
from sequence_ref import DT, EPS32, close, half_step, leaf
from test_gpu_sequence import gen, strided

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16", "f16"]
EPS = 1e-5


@pytest.fixture(scope="module")
def iga():
    import implicit_gemm_amd
    return implicit_gemm_amd


def layer_norm(h, w, b, eps=EPS):
    """(y, m, r) in 64 bits."""
    m = h.mean(-1)
    c = h - m[..., None]
    r = (c.pow(2).mean(-1) + eps).rsqrt()
    return c * r[..., None] * w + (b if b is not None else 0), m, r


def within(got, want, tol, what):
    bad = ~((got.double().cpu() - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d wrong, at %s" % (what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


# one row to many (teams of 256, 64 and 16 lanes), vectors cut short, the widest rows of each kernel
SHAPES = [(1, 1), (3, 7), (5, 64), (1, 257), (1100, 300), (1030, 1024), (2, 1537), (1025, 2048), (2, 4100), (3, 8192),
          (2, 16384), (0, 64), (1, 16383), (4096, 1), (4099, 96), (5000, 130), (4111, 255), (4100, 384), (4097, 385),
          (4098, 512), (4096, 513), (32769, 96), (32770, 130), (32768, 384)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_layer_norm_and_gradient(iga, rows, C, dtype):
    log("layer norm", rows, C, dtype)
    rand, dt = gen(rows * 31 + C), DT[dtype]
    x, res, dy, dh = (rand(rows, C, dtype=dt) for _ in range(4))
    w, b = rand(C), rand(C)
    if rows > 2:
        x[1] = 0
        res[1] = 0                      # no deviation: r = eps^-1/2, y = b
        x[2] = x[2] + 50                # a mean far above the deviation
    with_res, with_b = C % 2 == 0, C % 3 != 0
    b = b if with_b else None
    xd = strided(x, 3) if C < 5000 else x.cuda()
    wd, bd = w.cuda(), b.cuda() if with_b else None
    y, h, m, r = iga.layer_norm(xd, wd, bd, residual=res.cuda() if with_res else None, eps=EPS)
    hr = (x.double() + res.double()).to(dt) if with_res else x
    assert torch.equal(h.cpu(), hr)
    if not with_res:
        assert h is xd
    if rows == 0:
        assert y.shape == (0, C) and m.shape == r.shape == (0,)
        dx, dw, db = iga.layer_norm_grad(dy.cuda(), h, wd, m, r)
        assert dx.shape == (0, C) and not dw.any() and not db.any()
        return
    hl, wl, bl = leaf(hr), leaf(w), leaf(b)
    yr, mr, rr = layer_norm(hl, wl, bl)
    top = hr.double().abs().amax(1, keepdim=True)                 # of each row
    nr = ((hr.double() - mr.detach()[:, None]) * rr.detach()[:, None]).abs()
    dn = 72 * EPS32 * top * rr.detach()[:, None] + 40 * EPS32 * nr        # error of n
    mag = half_step(dt)
    wa = w.double().abs()
    within(m, mr.detach(), 72 * EPS32 * top[:, 0], "m")
    # r's own error: the squares' sum (72) and root, and m's error, which enters the squares to second order
    within(r, rr.detach(), rr.detach() * (60 * EPS32 + (72 * EPS32 * top[:, 0] * rr.detach()) ** 2), "r")
    dn2 = dn + nr * (72 * EPS32 * top * rr.detach()[:, None]) ** 2
    within(y, yr.detach(), mag * yr.detach().abs() + dn2 * wa + 2 * EPS32 * yr.detach().abs() + torch.finfo(dt).tiny, "y")
    g = (dy.double() * w.double()).abs()
    gmax = g.amax(1, keepdim=True)
    nmax, dnmax = nr.amax(1, keepdim=True), dn2.amax(1, keepdim=True)
    # g - mean(g) - n mean(g n): sums of 72 roundings, and n's error in both of its places
    slack = rr.detach()[:, None] * (80 * EPS32 * (g + gmax) + (nr + 1) * gmax * (140 * EPS32 * nmax + 2 * dnmax) + dn2 * gmax * nmax)
    for dhx in (None, dh):
        dx, dw, db = iga.layer_norm_grad(strided(dy, 5), h, wd, m, r, dh=dhx.cuda() if dhx is not None else None, bias=with_b)
        dxr, dwr, dbr = ref.grads((yr,), (dy.double(),), (hl, wl, bl))
        if dhx is not None:
            dxr = dxr + dhx.double()
        within(dx, dxr, mag * dxr.abs() + slack + 4 * EPS32 * dxr.abs() + torch.finfo(dt).tiny, "dx")
        terms = dy.double().abs()
        chain = (rows + 64) * EPS32
        within(dw, dwr, (terms * dn2).sum(0) + chain * (terms * nr).sum(0), "dw")
        assert (db is None) == (not with_b)
        if with_b:
            within(db, dbr, chain * terms.sum(0), "db")
        yr, _, _ = layer_norm(hl, wl, bl)


def test_gradient_against_differences(iga):
    """The gradient of a plain sum against the change of the outputs themselves, at full precision."""
    rand = gen(5)
    x, w, b, dy = rand(7, 33).double(), rand(33).double(), rand(33).double(), rand(7, 33).double()

    def loss(xx, ww, bb):
        return float((layer_norm(xx, ww, bb)[0] * dy).sum())

    xd = x.float().cuda()
    y, h, m, r = iga.layer_norm(xd, w.float().cuda(), b.float().cuda())
    dx, dw, db = iga.layer_norm_grad(dy.float().cuda(), h, w.float().cuda(), m, r)
    step = 1e-6
    for i, j in ((0, 0), (3, 17), (6, 32)):
        e = torch.zeros_like(x)
        e[i, j] = step
        # differences in 64 bits are good to step^2 of the third derivative and 1e-16 / step: 1e-8 here
        assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * step) - float(dx[i, j])) < 1e-4
        assert abs((loss(x, w + e[i], b) - loss(x, w - e[i], b)) / (2 * step) - float(dw[j])) < 1e-4
        assert abs((loss(x, w, b + e[i]) - loss(x, w, b - e[i])) / (2 * step) - float(db[j])) < 1e-4


def test_nan_and_infinity_stay_in_their_row(iga):
    x = torch.ones(5000, 256)
    x[:, ::2] = -1
    x[0, 5] = float("nan")
    x[1, 7] = float("inf")
    w, dy = torch.ones(256).cuda(), torch.ones(5000, 256).cuda()
    y, h, m, r = iga.layer_norm(x.cuda(), w, w)
    assert y[0].isnan().all() and y[1].isnan().all() and bool(torch.isfinite(y[2:]).all())
    dx = iga.layer_norm_grad(dy, h, w, m, r)[0]
    assert dx[0].isnan().all() and dx[1].isnan().all() and bool(torch.isfinite(dx[2:]).all())


def test_higher_rank_and_refusals(iga):
    rand = gen(1)
    x, w = rand(2, 3, 5, 64).cuda(), rand(64).cuda()
    y, _, m, r = iga.layer_norm(x, w, w)
    assert y.shape == x.shape and m.shape == r.shape == (2, 3, 5)
    assert torch.equal(y.view(-1, 64), iga.layer_norm(x.view(-1, 64), w, w)[0])
    assert torch.equal(iga.layer_norm(x[0, 0, 0], w, w)[0], y[0, 0, 0])
    for bad in (lambda: iga.layer_norm(x.transpose(0, 1), w), lambda: iga.layer_norm(x.transpose(2, 3), w),
                lambda: iga.layer_norm(x, w.bfloat16()), lambda: iga.layer_norm(x, w[:32]),
                lambda: iga.layer_norm(x, w, w[:32]), lambda: iga.layer_norm(x, w, residual=x[0]),
                lambda: iga.layer_norm(x.double(), w), lambda: iga.layer_norm(x, w.cpu()),
                lambda: iga.layer_norm(x, w, eps=-1.0), lambda: iga.layer_norm_grad(x, x, w, m[0], r),
                lambda: iga.layer_norm_grad(x, x, w, m, r[0]), lambda: iga.layer_norm_grad(x[0], x, w, m, r)):
        with pytest.raises((ValueError, TypeError, iga.ConvWgradError)):
            bad()


def test_runs_repeat_bit_for_bit_on_any_stream_and_in_a_graph(iga):
    rand = gen(9)
    x, res, dy = (rand(5000, 200, dtype=torch.bfloat16).cuda() for _ in range(3))
    w, b = rand(200).cuda(), rand(200).cuda()

    def step():
        y, h, m, r = iga.layer_norm(x, w, b, residual=res)
        return (y, h) + iga.layer_norm_grad(dy, h, w, m, r, dh=dy)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, m, r = iga.layer_norm(x, w, b, residual=res, stream=side)
    got = (y, h) + iga.layer_norm_grad(dy, h, w, m, r, dh=dy, stream=side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        x.copy_(gen(100 + seed)(5000, 200, dtype=torch.bfloat16))
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(eager, out))


def test_more_rows_than_workgroups_past_4_gib(iga):
    """2^20 + 5 rows of 4112 bytes, more than there are workgroups at most, against a part of themselves."""
    R, C = (1 << 20) + 5, 2056
    x = torch.randn(R, C, device="cuda", dtype=torch.bfloat16)
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    y, h, m, r = iga.layer_norm(x, w, b)
    dx, dw, db = iga.layer_norm_grad(y, h, w, m, r)
    for part in (slice(0, 3), slice(R - 7, R)):
        y1, _, m1, r1 = iga.layer_norm(x[part], w, b)
        assert torch.equal(y[part], y1) and torch.equal(m[part], m1) and torch.equal(r[part], r1)
        dx1 = iga.layer_norm_grad(y[part], x[part], w, m1, r1)[0]
        # the two calls' teams are of other sizes and add s1 and s2 in another order: a step of dx's type at most
        top = dx1.float().abs().amax(1, keepdim=True)
        assert bool(((dx[part].float() - dx1.float()).abs() <= 2 * half_step(torch.bfloat16) * top).all())
    want = torch.zeros(C, dtype=torch.float64, device="cuda")
    for i in range(0, R, 1 << 17):
        want += y[i:i + (1 << 17)].double().sum(0)
    # random signs: the partial sums' roundings stay below 2^-24 of the largest of them, which is under 8 sqrt(rows) times
    # the values' deviation, for each of a lane's 1025 additions and the 1024 joins
    size = 8 * R ** 0.5 * y[:4096].double().std(0) + want.abs()
    assert bool(((db.double() - want).abs() <= 2050 * EPS32 * size).all())

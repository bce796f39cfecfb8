"""Layer norm of rows whose mean lies far above their deviation, and its gradient, against the definition in 64 bits.

Tolerances.  A row's sum passes through at most 64 additions a lane and 8 between lanes: the first mean is off by up to 72
eps of the row's largest |h|, and that of what it leaves, whose terms are at most D = max |h - m| and that error, by 72 eps
of those.  So n = (h - m) r is off by dn = r (80 eps D + (72 eps)^2 top) beside some 40 roundings of n itself, whatever the
mean, where the first sum alone would leave 72 eps top r.  The stored m has one rounding more; the gradient has h and that m,
which is off by eps top at most, and finds the rest of it with the same error."""
import pytest
import torch

import sequence_ref as ref
from gpu_util import log
from sequence_ref import DT, EPS32, half_step, leaf
from test_gpu_layer_norm import EPS, iga, layer_norm, within  # noqa: F401
from test_gpu_sequence import gen

pytestmark = pytest.mark.gpu

# every team of lanes, forward and gradient, with whole vectors and with vectors cut short
SHAPES = [(7, 64), (6, 1537), (9, 4100), (5, 8192), (6, 16384), (5, 16383), (1100, 300), (1030, 1024), (4100, 96), (4099, 130),
          (32770, 96), (32769, 130), (4097, 385), (1, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_a_mean_far_above_the_deviation(iga, rows, C, dtype):  # noqa: F811
    log("layer norm of far means", rows, C, dtype)
    rand, dt = gen(rows * 17 + C), DT[dtype]
    x, dy, w, b = rand(rows, C), rand(rows, C, dtype=dt), rand(C), rand(C)
    kinds = [lambda t: 0 * t + 10000.1, lambda t: 1000 + 0.01 * t, lambda t: -30000.0 + t, lambda t: 0 * t - 1000.1,
             lambda t: 50 + t, lambda t: 3e-3 + 1e-6 * t]
    if dt != torch.float16:
        kinds += [lambda t: 1e6 + t, lambda t: 0 * t + 123456.7]
    for i, f in enumerate(kinds):
        x[i::len(kinds)] = f(x[i::len(kinds)])
    x = x.to(dt)
    wd = w.cuda()
    y, h, m, r = iga.layer_norm(x.cuda(), wd, b.cuda())
    hl, wl, bl = leaf(x), leaf(w), leaf(b)
    yr, mr, rr = layer_norm(hl, wl, bl, EPS)
    hd, mv, rv = x.double(), mr.detach()[:, None], rr.detach()[:, None]
    top, D, nr = hd.abs().amax(1, keepdim=True), (hd - mv).abs().amax(1, keepdim=True), ((hd - mv) * rv).abs()
    dm = 80 * EPS32 * D + (72 * EPS32) ** 2 * top
    within(m, mr.detach(), (dm + EPS32 * top)[:, 0], "m")
    # one error of the mean enters the squares to second order; their sum and its root have 72 roundings and some
    within(r, rr.detach(), (rv * (60 * EPS32 + (dm * rv) ** 2))[:, 0], "r")
    dn = dm * rv + 40 * EPS32 * nr + nr * (dm * rv) ** 2
    wa, mag, tiny = w.double().abs(), half_step(dt), torch.finfo(dt).tiny
    within(y, yr.detach(), mag * yr.detach().abs() + dn * wa + 2 * EPS32 * yr.detach().abs() + tiny, "y")
    dx, dw, db = iga.layer_norm_grad(dy.cuda(), h, wd, m, r)
    dxr, dwr, dbr = ref.grads((yr,), (dy.double(),), (hl, wl, bl))
    g = (dy.double() * w.double()).abs()
    gmax, nmax, dnmax = g.amax(1, keepdim=True), nr.amax(1, keepdim=True), dn.amax(1, keepdim=True)
    slack = rv * (80 * EPS32 * (g + gmax) + (nr + 1) * gmax * (140 * EPS32 * nmax + 2 * dnmax) + dn * gmax * nmax)
    within(dx, dxr, mag * dxr.abs() + slack + 4 * EPS32 * dxr.abs() + tiny, "dx")
    terms, chain = dy.double().abs(), (rows + 64) * EPS32
    within(dw, dwr, (terms * dn).sum(0) + chain * (terms * nr).sum(0), "dw")
    within(db, dbr, chain * terms.sum(0), "db")


def test_a_row_of_one_value_is_the_bias(iga):  # noqa: F811
    """h - m is zero: y = b and m = h to the last bit, whatever the value and the number of channels."""
    for C in (64, 130, 1000, 1537, 4099, 16383):
        for rows in (3, 5000):
            if rows * C > 1 << 24:
                continue
            value = torch.tensor([10000.1, -1000.1, 3.3e-5] * rows)[:rows]
            w, b = gen(C)(C).cuda(), gen(C + 1)(C).cuda()
            y, _, m, r = iga.layer_norm(value[:, None].expand(rows, C).contiguous().cuda(), w, b)
            assert torch.equal(m.cpu(), value) and torch.equal(y, b.expand(rows, C))

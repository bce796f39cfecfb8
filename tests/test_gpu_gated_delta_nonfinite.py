"""What an element that is not finite reaches in the gated delta rule, input by input: everything else stays as it is to the
last bit."""
import pytest
import torch

from gpu_util import log
from sequence_ref import DT
from test_gpu_gated_delta import iga, make  # noqa: F401

pytestmark = pytest.mark.gpu

OFF, HK, H, DK, DV = [0, 70, 200, 231], 2, 4, 64, 32
T, HEAD, KEY, COL = 133, 2, 1, 5          # a token of the second sequence's first chunk but one, a head and its key head
NAMES = ("q", "k", "v", "g", "beta", "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("what", NAMES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_it_reaches(iga, what, value, dtype):  # noqa: F811
    log("delta not finite", what, value, dtype)
    dt = DT[dtype]
    rand = torch.Generator().manual_seed(7)
    ins = dict(zip(NAMES, (*make(21, (OFF[-1],), HK, H, DK, DV, dt), torch.randn(3, H, DK, DV, generator=rand))))
    do = torch.randn(OFF[-1], H, DV, generator=rand).to(dt).cuda()
    off = torch.tensor(OFF, dtype=torch.int32).cuda()

    def call(x):
        x = {n: t.cuda() for n, t in x.items()}
        rows = [x[n] for n in NAMES[:5]]
        o, last, saved = iga.gated_delta(*rows, offsets=off, state=x["state"], save=True)
        d = iga.gated_delta_grad(do, *rows, saved, offsets=off, state=x["state"])
        return o.cpu(), last.cpu(), [t.cpu() for t in d]

    o, last, d = call(ins)
    bad = {n: t.clone() for n, t in ins.items()}
    at = {"q": (T, KEY, 3), "k": (T, KEY, 3), "v": (T, HEAD, COL), "g": (T, HEAD), "beta": (T, HEAD), "state": (1, HEAD, 3, COL)}
    bad[what][at[what]] = value
    ob, lastb, db = call(bad)
    heads = slice(2, 4) if what in "qk" else slice(HEAD, HEAD + 1)
    cols = slice(COL, COL + 1) if what in ("v", "state") else slice(None)
    begin = OFF[1] if what == "state" else T
    end = T + 1 if what == "q" else OFF[2]
    assert not torch.isfinite(ob[begin:end, heads, cols]).any()
    before = 0 if what in ("q", "state") else 63
    same = torch.ones_like(o, dtype=torch.bool)
    same[max(begin - before, OFF[1]):end, heads, cols] = False
    assert torch.equal(ob[same], o[same])
    same = torch.ones_like(last, dtype=torch.bool)
    if what != "q":
        assert not torch.isfinite(lastb[1, heads, :, cols]).any()
        same[1, heads, :, cols] = False
    assert torch.equal(lastb[same], last[same])
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), d, db):
        rows = torch.ones(a.shape[:2], dtype=torch.bool)
        if n == "dstate":
            rows[1, heads] = False
        else:
            rows[OFF[1]:OFF[2], KEY if n in ("dq", "dk") else heads] = False
        assert torch.equal(a[rows], b[rows]), n

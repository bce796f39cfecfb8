"""How accurate the gated delta rule's results are: 32 bits for every element type, over one chunk of tokens and over
thousands, with bounds that 16 bits do not keep (test_delta_pieces_cpu.py)."""
import pytest
import torch

import delta_pieces as dp
import delta_ref
from gpu_util import log
from sequence_ref import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def iga():
    import implicit_gemm_amd
    return implicit_gemm_amd


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", dp.CASES)
def test_results_have_32_bits(iga, case, dtype):
    log("delta accuracy", case, dtype)
    lens, Hk, H, Dk, Dv, kind = case
    dt = DT[dtype]
    ins, do, dlast = dp.inputs(case, dt)
    want = dp.reference(case, ins, do, dlast)
    size = dp.sizes(case, ins, do, want)
    three = dp.emulated(case, ins, do, dlast, 3, 3)
    *rows, state = (t.cuda() for t in ins)
    off = None
    if len(set(lens)) == 1:
        rows, do = [t.unflatten(0, (len(lens), -1)) for t in rows], do.unflatten(0, (len(lens), -1))
    else:
        off = torch.tensor(dp.offsets(lens), dtype=torch.int32).cuda()
    o, last, saved = iga.gated_delta(*rows, offsets=off, state=state, save=True)
    d = iga.gated_delta_grad(do.cuda(), *rows, saved, offsets=off, state=state, dstate_out=dlast.cuda())
    got = dict(zip(dp.NAMES, (o, last, *d)))
    got = {n: t if n in ("state", "dstate") or off is not None else t.flatten(0, 1) for n, t in got.items()}
    bound = dp.error_bounds(dp.errors(three, want, size))
    have = dp.errors(got, want, size)
    for n in dp.NAMES:
        if dt != torch.float32 and n in ("o", "dq", "dk", "dv"):
            most = dp.neighbour_bound(dp.expected_neighbours(three[n], want[n], dt))
            wrong = dp.neighbours(got[n], want[n])
            assert wrong <= most, "%s: %d of %d are not the rounded result, %.0f are expected at most" % (n, wrong, want[n].numel(), most)
        else:
            assert have[n] <= bound[n], (n, have[n], bound[n])
    # each element, the gradients of shared keys among them
    c, chain = (Dk + 190) * -(-max(lens) // 64), -(-max(lens) // 64)
    for n in dp.NAMES:
        t = dt if n in ("o", "dq", "dk", "dv") else torch.float32
        count = c + Dk if n == "o" else c if n == "state" else (2 * c + Dv + 64) * (H // Hk if n in ("dq", "dk") else 1)
        top = delta_ref.dg_scale(want["o"], ins[2], want["dv"], do.flatten(0, 1) if off is None else do, want["dg"]) if n == "dg" else None
        delta_ref.close(got[n], want[n], t, count, chain, n, scale=top)

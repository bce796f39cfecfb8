"""Calls of the gated delta rule that are refused, refused before anything of a wrong size is allocated."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def iga():
    import implicit_gemm_amd
    return implicit_gemm_amd


def test_queries_are_looked_at_before_states_are_allocated(iga):
    """A state that took its size from a wrong q would have 128 MB and more."""
    v, g = torch.zeros(2, 3, 8, 128).cuda(), torch.zeros(2, 3, 8).cuda()
    wrong = [torch.zeros(2, 3, 1 << 14).cuda(), torch.zeros(2, 3, 1, 1 << 14).cuda(), torch.zeros(2, 3, 3, 1 << 14).cuda(),
             torch.zeros(1 << 14).cuda(), torch.tensor(1.0).cuda(), torch.zeros(2, 3, 0, 64).cuda()]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for q in wrong:
        with pytest.raises((ValueError, iga.ConvWgradError)):
            iga.gated_delta(q, q, v, g, g)
    packed = v.flatten(0, 1)
    off = torch.tensor([0, 2, 6], dtype=torch.int32).cuda()
    for q in (torch.zeros(6, 1 << 14).cuda(), torch.zeros(6, 1, 1 << 14).cuda()):
        with pytest.raises((ValueError, iga.ConvWgradError)):
            iga.gated_delta(q, q, packed, g.flatten(0, 1), g.flatten(0, 1), offsets=off)
    assert torch.cuda.max_memory_allocated() <= before + (2 << 20)

"""Sequence operators without a GPU: argument errors of the C ABI (all before any launch), struct layouts, workspace
sizes, the cut of packed rows into pieces, and the 64-bit definitions against differences."""
import ctypes
import random

import pytest
import torch

import implicit_gemm_amd as iga
import sequence_ref as ref
from implicit_gemm_amd import sequence as sq

OK, NULL, SHAPE, DTYPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 5, 6, 7
P = 1 << 20     # a non-null pointer; nothing reads it before validation has passed


def test_struct_sizes_match_header_layout():
    view, tokens = 24, 40
    assert ctypes.sizeof(sq._View) == view and ctypes.sizeof(sq._Tokens) == tokens
    assert ctypes.sizeof(sq.NormArgs) == 104 and ctypes.sizeof(sq.NormGradArgs) == 104
    assert ctypes.sizeof(sq.ConvArgs) == tokens + 8 + 16 + view + 6 * 8 + view
    assert ctypes.sizeof(sq.ConvGradArgs) == 160 + 2 * view + 4 * 8
    assert ctypes.sizeof(sq.ScanArgs) == tokens + 16 + 16 + 8 + 5 * view + 16 + 3 * 8 + 4 * 8 + 8 + view
    assert ctypes.sizeof(sq.ScanGradArgs) == 304 + view + 10 * 8


def norm_args(**over):
    a = sq.NormArgs(4, 64, 1, 0, 1e-5, 0, P, 64, P, 64, P, P, P, P, P)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(channels=0), SHAPE), (dict(rows=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(group=128), SHAPE), (dict(channels=16385), UNSUPPORTED), (dict(dtype=7), DTYPE), (dict(x=0), NULL),
    (dict(w=0), NULL), (dict(y=0), NULL), (dict(residual=0), NULL), (dict(x=P + 1), MISALIGNED),
    (dict(w=P + 2), MISALIGNED), (dict(x_row=-64), SHAPE), (dict(rows=1 << 41), UNSUPPORTED),
])
def test_norm_refusals(over, status):
    assert sq._lib().seq_rms_norm(ctypes.byref(norm_args(**over)), None) == status
    assert sq._lib().seq_rms_norm(None, None) == NULL


@pytest.mark.parametrize("over,status", [(dict(group=100), SHAPE), (dict(group=-1), SHAPE), (dict(scale=0), NULL),
                                         (dict(group=512), SHAPE)])
def test_norm_e4m3_refusals(over, status):
    assert sq._lib().seq_rms_norm_e4m3(ctypes.byref(norm_args(**over)), None) == status


def test_norm_grad_refusals():
    lib = sq._lib()

    def args(**over):
        a = sq.NormGradArgs(4, 64, 1, 0, P, 64, P, 64, 0, 0, P, P, P, P)
        for k, v in over.items():
            setattr(a, k, v)
        return ctypes.byref(a)

    n = ctypes.c_size_t(0)
    assert lib.seq_rms_norm_grad_workspace(args(), ctypes.byref(n)) == OK and n.value == 64 * 4
    assert lib.seq_rms_norm_grad_workspace(args(), None) == NULL
    assert lib.seq_rms_norm_grad(args(), P, n.value - 1, None) == WORKSPACE
    assert lib.seq_rms_norm_grad(args(), None, n.value, None) == NULL
    assert lib.seq_rms_norm_grad(args(), P + 4, n.value, None) == MISALIGNED
    for over, status in ((dict(dw=0), NULL), (dict(h=0), NULL), (dict(rstd=0), NULL), (dict(dtype=3), DTYPE),
                         (dict(channels=0), SHAPE), (dict(dh_row=-1), SHAPE), (dict(dy=P + 1), MISALIGNED),
                         (dict(channels=20000), UNSUPPORTED)):
        assert lib.seq_rms_norm_grad(args(**over), P, n.value, None) == status, over


def conv_args(**over):
    tokens = [2, 10, 0, 0, 2]
    for i, k in enumerate(("sequences", "rows", "offsets", "slots", "pool")):
        tokens[i] = over.pop(k, tokens[i])
    a = sq.ConvArgs(tuple(tokens), 8, 4, 0, 1, 0, (P, 80, 8), P, P, P, 24, 2 * P, 24, (P, 80, 8))
    for k, v in over.items():
        setattr(a, k, v)
    return a


CONV_BAD = [
    (dict(sequences=0), SHAPE), (dict(rows=-1), SHAPE), (dict(width=1), SHAPE), (dict(width=5), SHAPE),
    (dict(channels=0), SHAPE), (dict(dtype=-1), DTYPE), (dict(pool=1), SHAPE), (dict(slots=P, pool=0), SHAPE),
    (dict(w=0), NULL), (dict(x=sq._View(0, 80, 8)), NULL), (dict(x=sq._View(P, -1, 8)), SHAPE),
    (dict(x=sq._View(P + 2, 80, 8)), MISALIGNED), (dict(offsets=P + 2), MISALIGNED), (dict(state_out_stride=23), SHAPE),
    (dict(state=2 * P, state_stride=32), SHAPE), (dict(rows=1 << 30), UNSUPPORTED), (dict(channels=1 << 21, state_out=0), UNSUPPORTED),
    (dict(sequences=1 << 20, pool=1 << 20, rows=1 << 21), UNSUPPORTED), (dict(y=sq._View(0, 80, 8)), NULL),
]


@pytest.mark.parametrize("over,status", CONV_BAD)
def test_conv_refusals(over, status):
    assert sq._lib().seq_causal_conv(ctypes.byref(conv_args(**dict(over))), None) == status


def test_conv_step_and_grad_refusals():
    lib = sq._lib()
    assert lib.seq_causal_conv_step(ctypes.byref(conv_args()), None) == SHAPE             # ten tokens, not one
    assert lib.seq_causal_conv_step(ctypes.byref(conv_args(rows=1, offsets=P)), None) == SHAPE
    g = sq.ConvGradArgs(conv_args(), (P, 80, 8), 0, (P, 80, 8), P, P, 0)
    n = ctypes.c_size_t(0)
    assert lib.seq_causal_conv_grad_workspace(ctypes.byref(g), ctypes.byref(n)) == OK and n.value >= 8 * 5 * 4
    assert lib.seq_causal_conv_grad(ctypes.byref(g), P, n.value - 1, None) == WORKSPACE
    assert lib.seq_causal_conv_grad(ctypes.byref(g), None, 0, None) == NULL
    for name in ("dw",):
        h = sq.ConvGradArgs(conv_args(), (P, 80, 8), 0, (P, 80, 8), P, P, 0)
        setattr(h, name, 0)
        assert lib.seq_causal_conv_grad(ctypes.byref(h), P, n.value, None) == NULL
    h = sq.ConvGradArgs(conv_args(), (P + 1, 80, 8), 0, (P, 80, 8), P, P, 0)
    assert lib.seq_causal_conv_grad(ctypes.byref(h), P, n.value, None) == MISALIGNED


def test_conv_says_which_windows_its_gradient_reads():
    """A call with slots writes the new windows over those that the gradient needs: each of the two calls says so."""
    assert "causal_conv_grad reads the windows before" in iga.causal_conv.__doc__
    assert "as they were before causal_conv" in iga.causal_conv_grad.__doc__


def scan_args(**over):
    tokens = [2, 10, 0, 0, 2]
    for i, k in enumerate(("sequences", "rows", "offsets", "slots", "pool")):
        tokens[i] = over.pop(k, tokens[i])
    v, bc = (P, 80, 8), (P, 320, 32)
    a = sq.ScanArgs(tuple(tokens), 8, 2, 16, 0, 1, 0, 0, v, v, v, bc, bc, 16, 16, P, P, P, P, 128, P, 128, P, v)
    for k, val in over.items():
        setattr(a, k, val)
    return a


SCAN_BAD = [
    (dict(sequences=0), SHAPE), (dict(groups=3), SHAPE), (dict(groups=0), SHAPE), (dict(states=0), SHAPE),
    (dict(states=33), UNSUPPORTED), (dict(dtype=9), DTYPE), (dict(channels=0), SHAPE), (dict(A=0), NULL),
    (dict(u=sq._View(0, 80, 8)), NULL), (dict(B=sq._View(P, 320, -1)), SHAPE), (dict(B_group=-1), SHAPE),
    (dict(A=P + 2), MISALIGNED), (dict(z=sq._View(P + 2, 80, 8)), MISALIGNED), (dict(state_out_stride=127), SHAPE),
    (dict(rows=1 << 30), UNSUPPORTED), (dict(pool=1), SHAPE), (dict(save=P + 1), MISALIGNED),
    (dict(state=P, state_stride=256), SHAPE), (dict(y=sq._View(0, 80, 8)), NULL),
]


@pytest.mark.parametrize("over,status", SCAN_BAD)
def test_scan_refusals(over, status):
    assert sq._lib().seq_selective_scan(ctypes.byref(scan_args(**dict(over))), P, 1 << 30, None) == status


def test_scan_step_and_grad_refusals():
    lib = sq._lib()
    assert lib.seq_selective_scan_step(ctypes.byref(scan_args()), None) == SHAPE
    # one long sequence of few channels is split: its workspace is asked for and checked
    a = scan_args(rows=5000)
    n = ctypes.c_size_t(0)
    assert lib.seq_selective_scan_workspace(ctypes.byref(a), ctypes.byref(n)) == OK and n.value > 0
    assert lib.seq_selective_scan(ctypes.byref(a), P, n.value - 1, None) == WORKSPACE
    assert lib.seq_selective_scan(ctypes.byref(a), P + 8, n.value, None) == MISALIGNED
    assert lib.seq_selective_scan(ctypes.byref(a), None, n.value, None) == NULL
    assert lib.seq_selective_scan_save(ctypes.byref(a), ctypes.byref(n)) == OK
    assert n.value == 2 * ((5000 + 15) // 16) * 8 * 16 * 4

    def grad(**over):
        g = sq.ScanGradArgs(scan_args(), (P, 80, 8), 0, *([P] * 9))
        for k, v in over.items():
            setattr(g, k, v)
        return ctypes.byref(g)

    assert lib.seq_selective_scan_grad_workspace(grad(), ctypes.byref(n)) == OK and n.value > 0
    assert lib.seq_selective_scan_grad(grad(), P, n.value - 1, None) == WORKSPACE
    for over, status in ((dict(du=0), NULL), (dict(dz=0), NULL), (dict(dA=0), NULL), (dict(dB=P + 2), MISALIGNED),
                         (dict(dy=sq._View(0, 80, 8)), NULL), (dict(fwd=scan_args(save=0)), NULL),
                         (dict(fwd=scan_args(states=40)), UNSUPPORTED), (dict(dy=sq._View(P, 80, 1 << 26)), UNSUPPORTED)):
        assert lib.seq_selective_scan_grad(grad(**over), P, n.value, None) == status, over


def grad_of(tokens, channels, groups, states):
    row = sq._View(P, 0, channels)
    f = sq.ScanArgs((*tokens, 0, 0, tokens[0]), channels, groups, states, 1, 1, 0, 0, row, row, row, row, row, 0, 0, P, P, P,
                    0, 0, 0, 0, P, row)
    return sq.ScanGradArgs(f, row, 0, *([P] * 9))


@pytest.mark.parametrize("tokens,channels,groups,states", [
    ((1, (1 << 21) + 16), 4160, 1, 32),      # the fold of dB and dC: 65 channel blocks, 32 lanes an output of both
    ((1, (1 << 22) + 16), 8192, 1, 16),
    ((16, 0), 1 << 20, 1 << 20, 32),         # the sweep: a workgroup of 512 lanes a channel and sequence
])
def test_scan_gradient_too_large_for_one_of_its_launches(tokens, channels, groups, states):
    """Refused before anything is enqueued, not by the launch that it does not fit after others ran."""
    n = ctypes.c_size_t(0)
    g = grad_of(tokens, channels, groups, states)
    lib = sq._lib()
    assert lib.seq_selective_scan_grad_workspace(ctypes.byref(g), ctypes.byref(n)) == UNSUPPORTED
    assert lib.seq_selective_scan_grad(ctypes.byref(g), P, 1 << 62, None) == UNSUPPORTED
    assert lib.seq_selective_scan_workspace(ctypes.byref(g.fwd), ctypes.byref(n)) == OK
    half = grad_of((tokens[0], tokens[1] // 2) if tokens[1] else (tokens[0] // 4, 0), channels, groups, states)
    assert lib.seq_selective_scan_grad_workspace(ctypes.byref(half), ctypes.byref(n)) == OK


def test_scan_is_refused_for_its_own_launches_only():
    """The size of a join that many sequences do not have, or do not need, is no reason."""
    n = ctypes.c_size_t(0)
    lib = sq._lib()

    def args(sequences, rows, offsets=None, A=P):
        f = grad_of((sequences, rows), 4096, 1, 16).fwd
        f.tokens.offsets, f.A = offsets, A
        return ctypes.byref(f)

    assert lib.seq_selective_scan_step(args(1 << 14, 1, A=0), None) == NULL           # its size passes
    assert lib.seq_selective_scan_step(args(1 << 18, 1, A=0), None) == UNSUPPORTED
    assert lib.seq_selective_scan_workspace(args(1 << 14, 64), ctypes.byref(n)) == OK and n.value == 0
    # packed rows that would be split for a sequence of all of them: a join of 2^32 lanes, and the half of it
    assert lib.seq_selective_scan_workspace(args(1 << 14, 1 << 20, P), ctypes.byref(n)) == OK and n.value == 0
    assert lib.seq_selective_scan_workspace(args(1 << 13, 1 << 20, P), ctypes.byref(n)) == OK and n.value > 0
    assert lib.seq_selective_scan_workspace(args(1 << 20, 1 << 20, P), ctypes.byref(n)) == UNSUPPORTED


def test_a_forward_scan_needs_no_gradient_of_its_size():
    """The Python call asks for the gradient's workspace only when it computes one."""
    sizes = (1, (1 << 21) + 16, False, 4160, 1, 32, 1, 0)
    saved, space = sq._scan_space(*sizes)
    assert saved == ((1 << 17) + 1) * 4160 * 32 * 4 and space > 0
    with pytest.raises(iga.ConvWgradError):
        sq._scan_grad_space(*sizes)
    assert sq._scan_grad_space(1, 1 << 20, *sizes[2:])[1] > 0


def test_tensors_on_the_host_are_refused():
    x, w = torch.zeros(2, 8), torch.ones(8)
    with pytest.raises(ValueError):
        iga.rms_norm(x, w)
    with pytest.raises(ValueError):
        iga.causal_conv(torch.zeros(1, 2, 8), torch.zeros(8, 4))
    with pytest.raises(AttributeError):
        iga.no_such_operator


def find_piece(offsets, rows, shift, piece):
    """The kernels' search: (sequence, start, length, first token of the piece) or None."""
    S = len(offsets) - 1
    start = [min(max(o, 0), rows) for o in offsets]
    base = [(start[s] >> shift) + s for s in range(S + 1)]
    lo, n = 0, S + 1
    while n > 1:
        step = (n + 63) >> 6
        cnt = sum(lane * step < n and base[lo + lane * step] <= piece for lane in range(64))
        if cnt == 0:
            return None
        lo, n = lo + (cnt - 1) * step, min(step, n - (cnt - 1) * step)
    stop = start[lo + 1] if lo < S else rows
    length = max(stop - start[lo], 0)
    j = piece - base[lo]
    if j < 0 or (j > 0 and (j << shift) >= length):
        return None
    return lo, start[lo], length, j << shift


@pytest.mark.parametrize("seed", range(16))
def test_pieces_cover_packed_rows_once(seed):
    rng = random.Random(seed)
    S = 5000 if seed == 0 else rng.choice([1, 2, 7, 63, 64, 65, 130])
    lens = [rng.choice([0, 1, 2, 15, 16, 17, 100]) if rng.random() < 0.7 else rng.randint(0, 60) for _ in range(S)]
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    rows = offsets[-1] + rng.choice([0, 0, 1, 40])
    for shift in (4, 5, 30) if S < 5000 else (5,):
        seen, rows_seen = set(), 0
        pieces = (rows >> shift) + S + 1
        for p in range(pieces):
            got = find_piece(offsets, rows, shift, p)
            if got is None:
                continue
            s, start, length, t0 = got
            assert (s, t0) not in seen and 0 <= start + t0 <= rows
            assert length == (lens[s] if s < S else rows - offsets[-1])
            seen.add((s, t0))
            rows_seen += min(length - t0, 1 << shift)
            assert (start >> 4) + s + (t0 >> 4) < (rows >> 4) + S + 1        # where its states are saved
        assert rows_seen == rows
        assert {s for s, t0 in seen if t0 == 0} >= set(range(S))             # an empty sequence has a piece too


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [0, -5, 400, 3], [7, 7, 7, 7], [90, 60, 30, 0]])
def test_bad_offsets_stay_in_bounds(offsets):
    rows = 80
    for shift in (4, 6, 30):
        for p in range((rows >> shift) + len(offsets)):
            got = find_piece(offsets, rows, shift, p)
            if got:
                s, start, length, t0 = got
                assert 0 <= start and start + length <= rows or length == 0
                assert (start >> 4) + s + (max(length - 1, 0) >> 4) < (rows >> 4) + len(offsets)


def _difference(f, tensors, direction, eps=1e-5):
    hi = f(*[t + eps * d for t, d in zip(tensors, direction)])
    lo = f(*[t - eps * d for t, d in zip(tensors, direction)])
    return (hi - lo) / (2 * eps)


def test_definitions_against_differences():
    """The 64-bit gradients that the GPU tests compare with, against central differences (error eps^2)."""
    g = torch.Generator().manual_seed(5)

    def rand(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    T, D, N, G = 9, 4, 3, 2
    offsets = [0, 5, 5, 8]
    ins = [rand(T, D), rand(T, D) * 0.5, -rand(D, N).abs(), rand(T, G, N), rand(T, G, N), rand(D), rand(T, D), rand(D),
           rand(3, D, N)]
    sy, sh = rand(T, D), rand(3, D, N)

    def loss(u, d, A, B, C, skip, z, bias, state):
        y, h = ref.scan(u, d, A, B, C, skip, z, bias, True, offsets, state)
        return (y * sy).sum() + (h * sh).sum()

    leaves = [t.clone().requires_grad_(True) for t in ins]
    grads = torch.autograd.grad(loss(*leaves), leaves)
    direction = [rand(*t.shape) for t in ins]
    want = sum((a * b).sum() for a, b in zip(grads, direction))
    assert abs(_difference(loss, ins, direction) - want) <= 1e-7 * (1 + abs(want))

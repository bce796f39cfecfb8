"""The gated delta rule without a GPU: argument errors of the C entries (all before any launch), struct layouts, sizes,
and the definition against differences and against a plain chunked form."""
import ctypes

import pytest
import torch

import delta_ref
from implicit_gemm_amd import sequence as sq

OK, NULL, SHAPE, DTYPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 5, 6, 7
P = 1 << 20     # a non-null pointer; nothing reads it before validation has passed


def view(row=512, ptr=P):
    return sq._View(ptr, 8 * row, row)


def args(**over):
    a = sq.DeltaArgs()
    a.tokens = sq._Tokens(2, 8, 0, 0, 2)
    a.heads, a.key_heads, a.key_dim, a.value_dim, a.dtype, a.scale = 4, 2, 64, 32, 1, 0.125
    a.q, a.k, a.v, a.o, a.g, a.beta = view(), view(), view(), view(), view(4), view(4)
    a.q_head, a.k_head, a.v_head = 64, 64, 32
    a.state, a.state_out, a.state_stride, a.state_out_stride = P, P, 4 * 64 * 32, 4 * 64 * 32
    for name, v in over.items():
        if "__" in name:
            outer, inner = name.split("__")
            part = getattr(a, outer)
            setattr(part, inner, v)
        else:
            setattr(a, name, v)
    return a


def grad_args(fwd=None, **over):
    g = sq.DeltaGradArgs()
    g.fwd = fwd or args(save=P)
    g.dout, g.dout_head = view(), 32
    g.dq = g.dk = g.dv = g.dg = g.dbeta = P
    for name, v in over.items():
        if "__" in name:
            outer, inner = name.split("__")
            setattr(getattr(g, outer), inner, v)
        else:
            setattr(g, name, v)
    return g


def test_struct_sizes():
    view_size, tokens = 24, 40
    assert ctypes.sizeof(sq.DeltaArgs) == tokens + 16 + 16 + 3 * view_size + 24 + 2 * view_size + 4 * 8 + 8 + view_size
    assert ctypes.sizeof(sq.DeltaGradArgs) == 280 + view_size + 8 + 8 + 6 * 8


SHAPES = [
    (dict(heads=0), SHAPE), (dict(key_heads=0), SHAPE), (dict(key_heads=3), SHAPE), (dict(key_dim=0), SHAPE),
    (dict(value_dim=0), SHAPE), (dict(key_dim=257), UNSUPPORTED), (dict(value_dim=1025), UNSUPPORTED), (dict(dtype=9), DTYPE),
    (dict(heads=1 << 17, key_heads=1 << 17), UNSUPPORTED), (dict(q__row=-1), SHAPE), (dict(k__batch=-1), SHAPE),
    (dict(v__row=1 << 24), UNSUPPORTED), (dict(q__row=1 << 24), UNSUPPORTED), (dict(g__row=-1), SHAPE), (dict(q_head=-1), SHAPE),
    (dict(tokens__sequences=0), SHAPE), (dict(tokens__rows=-1), SHAPE), (dict(tokens__pool=1), SHAPE),
    (dict(tokens__rows=1 << 29, tokens__sequences=1 << 29, tokens__pool=1 << 29), UNSUPPORTED),
    (dict(tokens__rows=1 << 29), UNSUPPORTED), (dict(state_stride=-1), SHAPE), (dict(tokens__offsets=P + 2), MISALIGNED),
    (dict(heads=32768, key_heads=1, value_dim=1024), UNSUPPORTED)]
INPUTS = [(dict(q__ptr=0), NULL), (dict(k__ptr=0), NULL), (dict(v__ptr=0), NULL), (dict(g__ptr=0), NULL),
          (dict(beta__ptr=0), NULL), (dict(q__ptr=P + 1), MISALIGNED), (dict(g__ptr=P + 2), MISALIGNED),
          (dict(save=P + 8), MISALIGNED)]
FORWARD = [(dict(o__ptr=0), NULL), (dict(o__ptr=P + 1), MISALIGNED), (dict(o__row=1 << 24), UNSUPPORTED),
           (dict(state=P + 2), MISALIGNED), (dict(state_out_stride=100), SHAPE), (dict(state_stride=100), SHAPE),
           (dict(state_out=P + 2), MISALIGNED)]


@pytest.mark.parametrize("over,status", SHAPES + INPUTS + FORWARD)
def test_refusals(over, status):
    lib = sq._lib()
    assert lib.seq_gated_delta(ctypes.byref(args(**over)), P, 1 << 40, None) == status
    assert lib.seq_gated_delta(None, P, 1 << 40, None) == NULL


@pytest.mark.parametrize("over,status", [s for s in SHAPES if "tokens__rows" not in s[0]] + INPUTS + FORWARD)
def test_step_refusals(over, status):
    lib = sq._lib()
    a = args(**over)
    a.tokens.rows = 1
    assert lib.seq_gated_delta_step(ctypes.byref(a), None) == status
    for wrong in (dict(tokens__rows=2), dict(tokens__rows=1, tokens__offsets=P)):
        assert lib.seq_gated_delta_step(ctypes.byref(args(**wrong)), None) == SHAPE


@pytest.mark.parametrize("over,status", SHAPES + INPUTS + [(dict(save=0), NULL)])
def test_gradient_refuses_what_the_forward_does(over, status):
    fwd = args(**{"save": P, **over})
    assert sq._lib().seq_gated_delta_grad(ctypes.byref(grad_args(fwd)), P, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(dout__ptr=0), NULL), (dict(dq=0), NULL), (dict(dk=0), NULL), (dict(dv=0), NULL), (dict(dg=0), NULL),
    (dict(dbeta=0), NULL), (dict(dout__ptr=P + 1), MISALIGNED), (dict(dg=P + 2), MISALIGNED), (dict(dstate=P + 2), MISALIGNED),
    (dict(dstate_out=P + 1), MISALIGNED), (dict(dout_head=-1), SHAPE), (dict(dout__row=1 << 24), UNSUPPORTED)])
def test_gradient_refusals(over, status):
    assert sq._lib().seq_gated_delta_grad(ctypes.byref(grad_args(**over)), P, 1 << 40, None) == status


def test_sizes():
    lib, n = sq._lib(), ctypes.c_size_t(0)
    for f, a in ((lib.seq_gated_delta_save, args()), (lib.seq_gated_delta_workspace, args()),
                 (lib.seq_gated_delta_grad_workspace, grad_args())):
        assert f(None, ctypes.byref(n)) == NULL and f(ctypes.byref(a), None) == NULL
        assert f(ctypes.byref(a), ctypes.byref(n)) == OK and n.value > 0
    assert lib.seq_gated_delta_workspace(ctypes.byref(args()), ctypes.byref(n)) == OK
    for ptr, size, status in ((0, n.value, NULL), (P, n.value - 1, WORKSPACE), (P + 4, n.value, MISALIGNED)):
        assert lib.seq_gated_delta(ctypes.byref(args()), ptr, size, None) == status
    assert lib.seq_gated_delta_grad_workspace(ctypes.byref(grad_args()), ctypes.byref(n)) == OK
    for ptr, size, status in ((0, n.value, NULL), (P, n.value - 1, WORKSPACE), (P + 4, n.value, MISALIGNED)):
        assert lib.seq_gated_delta_grad(ctypes.byref(grad_args()), ptr, size, None) == status


def inputs(T=90, H=2, Dk=6, Dv=5):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k = (t / t.norm(dim=-1, keepdim=True) for t in (r(1, T, 1, Dk), r(1, T, 1, Dk)))
    return [q, k, r(1, T, H, Dv), -r(1, T, H).abs() * 0.2, torch.sigmoid(r(1, T, H))]


def test_definition_against_differences():
    ins = [t.requires_grad_(True) for t in inputs(T=12)]
    state = torch.randn(1, 2, 6, 5, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(lambda *a: delta_ref.delta(*a[:5], state=a[5]), (*ins, state))


def test_definition_against_the_triangular_system():
    """A chunk's tokens as one system: (1 + M) Z = V - e^G (K S), as the kernels solve it."""
    q, k, v, g, beta = (t[0] for t in inputs(T=64, H=1))
    o, last = delta_ref.delta(q[None], k[None], v[None], g[None], beta[None])
    q, k, v, g, beta = q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]
    G = g.cumsum(0)
    e = torch.exp(G[:, None] - G[None, :]).tril()
    M = ((k @ k.T) * e).tril(-1) * beta
    Z = torch.linalg.solve_triangular(torch.eye(64, dtype=torch.float64) + M, v, upper=False, unitriangular=True)
    want = ((q @ k.T) * e * beta) @ Z * 6 ** -0.5
    assert torch.allclose(o[0, :, 0], want, atol=1e-12)
    assert torch.allclose(last[0, 0], (k * (beta * torch.exp(G[-1] - G))[:, None]).T @ Z, atol=1e-12)


def block_rows(r, lower):
    return [s for s in range(2) if (s <= r // 2 if lower else s >= r // 2)]


def test_the_blocks_of_a_triangle_have_places_of_their_own():
    """The operand blocks of a lower and an upper triangular 64 x 64 matrix, numbered as the kernels number them."""
    lower = [r if r < 2 else 2 * r - 2 + s for r in range(4) for s in block_rows(r, True)]
    upper = [2 * r + s if r < 2 else r + 2 for r in range(4) for s in block_rows(r, False)]
    assert sorted(lower) == sorted(upper) == list(range(6))

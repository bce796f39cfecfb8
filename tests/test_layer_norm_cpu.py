"""Layer norm without a GPU: argument errors of the C entries (all before any launch), struct layouts, workspace sizes."""
import ctypes

import pytest

from implicit_gemm_amd import sequence as sq

OK, NULL, SHAPE, DTYPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 5, 6, 7
P = 1 << 20     # a non-null pointer; nothing reads it before validation has passed


def args(**over):
    a = sq.LayerNormArgs(4, 64, 1, 1e-5, P, 64, P, 64, P, P, P, P, P, P)
    for k, v in over.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def grad_args(**over):
    a = sq.LayerNormGradArgs(4, 64, 1, 0, P, 64, P, 64, 0, 0, P, P, P, P, P, P)
    for k, v in over.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_struct_sizes():
    assert ctypes.sizeof(sq.LayerNormArgs) == 16 + 8 + 10 * 8
    assert ctypes.sizeof(sq.LayerNormGradArgs) == 16 + 8 + 12 * 8


@pytest.mark.parametrize("over,status", [
    (dict(channels=0), SHAPE), (dict(rows=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(channels=16385), UNSUPPORTED), (dict(rows=1 << 41), UNSUPPORTED), (dict(dtype=7), DTYPE), (dict(x=0), NULL),
    (dict(w=0), NULL), (dict(y=0), NULL), (dict(residual=0), NULL), (dict(x=P + 1), MISALIGNED), (dict(w=P + 2), MISALIGNED),
    (dict(b=P + 1), MISALIGNED), (dict(mean=P + 2), MISALIGNED), (dict(rstd=P + 2), MISALIGNED), (dict(h=P + 1), MISALIGNED),
    (dict(x_row=-64), SHAPE), (dict(residual_row=-1), SHAPE)])
def test_refusals(over, status):
    assert sq._lib().seq_layer_norm(args(**over), None) == status
    assert sq._lib().seq_layer_norm(None, None) == NULL


@pytest.mark.parametrize("over,status", [
    (dict(channels=0), SHAPE), (dict(rows=-1), SHAPE), (dict(channels=16385), UNSUPPORTED), (dict(dtype=7), DTYPE),
    (dict(dy=0), NULL), (dict(h=0), NULL), (dict(mean=0), NULL), (dict(rstd=0), NULL), (dict(dx=0), NULL), (dict(dw=0), NULL),
    (dict(w=0), NULL), (dict(dy=P + 1), MISALIGNED), (dict(dh=P + 1), MISALIGNED), (dict(db=P + 2), MISALIGNED),
    (dict(mean=P + 1), MISALIGNED), (dict(dy_row=-1), SHAPE), (dict(dh_row=-1), SHAPE)])
def test_gradient_refusals(over, status):
    n = ctypes.c_size_t(0)
    assert sq._lib().seq_layer_norm_grad_workspace(grad_args(), ctypes.byref(n)) == OK and n.value > 0
    assert sq._lib().seq_layer_norm_grad(grad_args(**over), P, 1 << 30, None) == status


def test_gradient_workspace():
    lib, n = sq._lib(), ctypes.c_size_t(0)
    assert lib.seq_layer_norm_grad_workspace(None, ctypes.byref(n)) == NULL
    assert lib.seq_layer_norm_grad_workspace(grad_args(), None) == NULL
    assert lib.seq_layer_norm_grad_workspace(grad_args(rows=1 << 39), ctypes.byref(n)) == OK
    assert n.value <= 1024 * 2 * 64 * 4           # does not grow with the rows
    assert lib.seq_layer_norm_grad_workspace(grad_args(), ctypes.byref(n)) == OK
    assert lib.seq_layer_norm_grad(grad_args(), 0, n.value, None) == NULL
    assert lib.seq_layer_norm_grad(grad_args(), P, n.value - 1, None) == WORKSPACE
    assert lib.seq_layer_norm_grad(grad_args(), P + 4, n.value, None) == MISALIGNED

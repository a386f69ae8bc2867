"""Refusals of the operators around the layer (no GPU): the C entry points check
their arguments before any device call, the Python functions before the C call."""
import ctypes

import pytest
import torch

import moe_megakernel_b200 as mk

BF = torch.bfloat16
A = ctypes.c_void_p(1 << 20)        # an aligned address that no refused call may touch
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    from moe_megakernel_b200 import build, load_library
    build.build()
    return load_library()


def _coeffs(n=3):
    return (ctypes.c_float * n)(*([1.0] * n))


GROUPED = dict(x=A, ldx=64, W=A, offsets=A, rows=10, groups=4, K=64, N=128, transpose=0, dtype=0, y=A, ldy=128,
               error_word=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(x=ODD), 1), (dict(W=None), 1), (dict(W=ODD), 1), (dict(offsets=None), 1),
    (dict(y=None), 1), (dict(y=ODD), 1), (dict(rows=-1), 1), (dict(groups=0), 1), (dict(groups=1025), 2),
    (dict(K=60, ldx=64), 2), (dict(N=100), 2), (dict(K=0), 2), (dict(ldx=56), 1), (dict(ldx=68), 1), (dict(ldy=120), 1),
    (dict(rows=(1 << 30) + 1), 2), (dict(dtype=2), 1), (dict(dtype=7), 1), (dict(error_word=ctypes.c_void_p(6)), 1)])
def test_grouped_matmul_refusals(lib, change, status):
    assert lib.moe_grouped_matmul(*(GROUPED | change).values()) == status


WGRAD = dict(x=A, ldx=64, dy=A, lddy=128, offsets=A, rows=10, groups=4, K=64, N=128, dtype=0, dW=A, error_word=None,
             stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(dy=ODD), 1), (dict(dW=None), 1), (dict(dW=ODD), 1), (dict(offsets=None), 1),
    (dict(rows=-1), 1), (dict(groups=0), 1), (dict(groups=5000), 2), (dict(K=4), 2), (dict(lddy=100), 1),
    (dict(dtype=2), 1)])
def test_wgrad_refusals(lib, change, status):
    assert lib.moe_grouped_matmul_wgrad(*(WGRAD | change).values()) == status


LINEAR = dict(x=A, ldx=64, W=A, bias=None, residual=None, ldr=0, T=3, K=64, N=128, activation=0, dtype=0, y=A, ldy=128,
              preact=None, ldz=0, error_word=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(W=None), 1), (dict(y=None), 1), (dict(bias=ODD), 1), (dict(residual=A, ldr=64), 1),
    (dict(residual=ODD, ldr=128), 1), (dict(preact=A, ldz=0), 1), (dict(T=-1), 1), (dict(activation=5), 1),
    (dict(activation=-1), 1), (dict(dtype=2), 1), (dict(K=20), 2), (dict(N=4), 2),
    (dict(T=2 ** 31 - 1), 2)])
def test_linear_refusals(lib, change, status):
    assert lib.moe_linear(*(LINEAR | change).values()) == status


BACKWARD = dict(dy=A, lddy=128, x=A, ldx=64, W=A, preact=A, ldz=128, T=3, K=64, N=128, activation=2, dtype=0, dx=A,
                lddx=64, dW=A, dbias=A, workspace=A, workspace_bytes=1 << 20, error_word=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), 1), (dict(x=None), 1), (dict(W=None), 1), (dict(preact=None), 1), (dict(ldz=0), 1), (dict(dx=ODD), 1),
    (dict(dW=ODD), 1), (dict(dbias=ODD), 1), (dict(workspace=None), 1), (dict(workspace=ODD), 1),
    (dict(workspace_bytes=100), 3), (dict(lddx=8), 1), (dict(activation=9), 1), (dict(N=12), 2)])
def test_linear_backward_refusals(lib, change, status):
    assert lib.moe_linear_backward(*(BACKWARD | change).values()) == status


def test_linear_backward_workspace(lib):
    f = lib.moe_linear_backward_workspace_bytes
    assert f(0, 128, 2, 1) == 0 and f(10, 128, 0, 0) == 0
    assert f(10, 128, 2, 0) == 10 * 128 * 2            # dz alone
    assert f(10, 128, 0, 1) == 128 * 4                 # one chunk of column sums
    assert f(100000, 128, 0, 1) == 128 * 128 * 4       # at most 128 chunks


ORTHO = dict(G=A, ldg=40, bsg=40 * 30, batch=2, m=30, n=40, dtype=0, steps=1, coeffs=_coeffs(), eps=1e-7, out=A, ldo=40,
             bso=40 * 30, workspace=A, workspace_bytes=1 << 30, error_word=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(G=None), 1), (dict(out=None), 1), (dict(ldg=1 << 50), 1), (dict(G=ctypes.c_void_p((1 << 20) + 1)), 1), (dict(ldg=39), 1),
    (dict(ldo=8), 1), (dict(bsg=100), 1), (dict(bso=100), 1), (dict(batch=-1), 1), (dict(m=0), 1), (dict(dtype=1), 1),
    (dict(coeffs=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(steps=0), 2), (dict(steps=65), 2),
    (dict(m=70000, ldg=70000, bsg=1 << 40), 2), (dict(workspace=None), 1), (dict(workspace=ODD), 1),
    (dict(workspace_bytes=1000), 3)])
def test_orthogonalize_refusals(lib, change, status):
    assert lib.moe_orthogonalize(*(ORTHO | change).values()) == status


def test_orthogonalize_workspace(lib):
    f = lib.moe_orthogonalize_workspace_bytes
    assert f(0, 4, 4) == 0 and f(1, 0, 4) == 0
    one, two = f(1, 129, 250), f(2, 129, 250)
    assert one >= 2 * 129 * 256 * 2 + 129 * 256 + 2 * 129 * 192 * 2 and one % 256 == 0
    assert f(1, 250, 129) == one
    assert one < two <= 2 * one


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _off(*v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: mk.grouped_matmul(_z(4, 64), _z(2, 32, 64), _off(0, 2, 4)),                          # K differs
    lambda: mk.grouped_matmul(_z(4, 64), _z(3, 64, 32), _off(0, 2, 4)),                          # groups differ
    lambda: mk.grouped_matmul(_z(4, 64), _z(2, 64, 32), _off(0, 2, 4).long()),                   # offsets type
    lambda: mk.grouped_matmul(_z(4, 64), _z(2, 64, 32), _off(0)),                                # no group
    lambda: mk.grouped_matmul(_z(4, 64, dtype=torch.float32), _z(2, 64, 32), _off(0, 2, 4)),     # type
    lambda: mk.grouped_matmul(_z(4, 64), _z(2, 64, 32, dtype=torch.float16), _off(0, 2, 4)),     # mixed types
    lambda: mk.grouped_matmul(_z(64, 4).T, _z(2, 64, 32), _off(0, 2, 4)),                        # last index strided
    lambda: mk.grouped_matmul(_z(4, 64), _z(2, 64, 32), _off(0, 2, 4)),                          # not on a GPU
    lambda: mk.grouped_matmul_wgrad(_z(4, 64), _z(5, 32), _off(0, 2, 4)),
    lambda: mk.grouped_matmul_wgrad(_z(4, 64), _z(4, 32), _off(0, 2, 4)),
    lambda: mk.linear(_z(4, 64), _z(32, 64)),
    lambda: mk.linear(_z(4, 64), _z(64, 32), bias=_z(64)),
    lambda: mk.linear(_z(4, 64), _z(64, 32), residual=_z(4, 64)),
    lambda: mk.linear(_z(4, 64), _z(64, 32), activation="tanh"),
    lambda: mk.linear(_z(4, 64), _z(64, 32)),
    lambda: mk.linear_backward(_z(4, 32), _z(4, 64), _z(64, 32), activation="gelu"),              # no preact
    lambda: mk.linear_backward(_z(4, 64), _z(4, 64), _z(64, 32)),
    lambda: mk.linear_backward(_z(4, 32), _z(4, 64), _z(64, 32)),
    lambda: mk.orthogonalize(_z(4)),
    lambda: mk.orthogonalize(_z(4, 4, dtype=torch.float16)),
    lambda: mk.orthogonalize(_z(4, 4), steps=0),
    lambda: mk.orthogonalize(_z(4, 4), coeffs=(1.0, 2.0)),
    lambda: mk.orthogonalize(_z(4, 4), steps=3, coeffs=[(1.0, 2.0, 3.0)] * 2),
    lambda: mk.orthogonalize(_z(4, 6).T),
    lambda: mk.orthogonalize(_z(4, 4))])
def test_python_refusals(call):
    with pytest.raises(ValueError):
        call()


def test_python_refuses_other_objects():
    with pytest.raises(TypeError):
        mk.linear([[1.0]], _z(64, 32))
    with pytest.raises(TypeError):
        mk.orthogonalize(None)

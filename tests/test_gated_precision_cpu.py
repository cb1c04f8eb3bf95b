"""The bounds of the gated block's precision tests tell a value kept in two 16-bit
terms from one rounded once: both evaluated here, without a GPU."""
import pytest
import torch

import gated_exact as E

TYPES = [torch.bfloat16, torch.float16]
SIZES = [(70, 272, 512, 16), (130, 96, 1024, 128), (5, 16, 64, 16), (9, 500, 9088, 48)]


def terms(v, dt, n, k=2.0 ** -10):
    """v in n terms, by way of a power of two that leaves it in fp16's range."""
    out, rest = torch.zeros_like(v), v * k
    for _ in range(n):
        t = rest.to(dt).double()
        out, rest = out + t, rest - t
    return out / k


def passes(y, ref, err, dt):
    try:
        E.check(y.to(dt), ref, err, "")
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,N,K,r", SIZES)
def test_forward_bound(T, N, K, r, dt):
    s = 2.0 ** -8
    X, A, B = E.forward_case(T, N, K, r, 0, "cpu")
    assert all((t.to(dt).double() == t).all() for t in (X, *A, *B))
    for i, (ref, err) in enumerate(E.projections(X, A, B, s, dt)):
        u = X @ A[i].T
        assert (u.float().double() == u).all()
        assert passes(s * terms(u, dt, 2) @ B[i].T, ref, err, dt)
        assert not passes(terms(s * u, dt, 1) @ B[i].T, ref, err, dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,N,K,r", SIZES)
def test_dx_bound(T, N, K, r, dt):
    s = 2.0 ** -12
    dH, A, B, P = E.backward_case(T, N, K, r, 0, "cpu")
    ref, err = E.dx(dH, A, B, P, s, dt)
    for n in (1, 2):
        val = sum(s * terms((dH * p) @ b, dt, n) @ a for p, a, b in zip(P[::-1], A, B))
        assert passes(val, ref, err, dt) == (n == 2)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,N,K,r", [c for c in SIZES if c[1] > 16])
def test_da_bound(T, N, K, r, dt):
    """G in as many terms as its bits need, and in one fewer."""
    dH, A, B, P = E.backward_case(T, N, K, r, 0, "cpu")
    X = E.pairs(torch.Generator().manual_seed(1), K, T, "cpu").T
    need = 3 if dt == torch.bfloat16 else 2
    for i, (ref, err) in enumerate(E.da(dH, X, B, P, 0.25, dt)):
        for n in (need - 1, need):
            y = (0.25 * terms((dH * P[1 - i]) @ B[i], dt, n).T @ X).float()
            assert passes(y, ref, err, torch.float32) == (n == need)


@pytest.mark.parametrize("dt", TYPES)
def test_picked_bound(dt):
    """Every term of d, and one fewer: dA and dB with their last term lost."""
    T, N, K, r = 48, 272, 320, 48
    dH, P, U, B, X, d = E.picked_case(T, N, K, r, 0, "cpu", dt)
    need = 3 if dt == torch.bfloat16 else 2
    for v, ((dA, eA), (dB, eB)) in zip(d, E.picked(d, r, K, dt)):
        assert torch.equal(dA, (v @ B).T @ X) and torch.equal(dB, v.T @ U)
        for n in (need - 1, need):
            t = terms(v, dt, n, 2.0 ** 14)
            assert passes(t.T @ U, dB, eB, torch.float32) == (n == need)
            assert passes((t @ B).T @ X, dA, eA, torch.float32) == (n == need)

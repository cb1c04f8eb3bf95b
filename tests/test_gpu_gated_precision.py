"""How much of U = X A^T and of G = d B the gated block's adapters keep, and over
which range: bounds per element that leave no room for one 16-bit rounding."""
import pytest
import torch

import gated_exact as E
from gpu_util import dev
from test_gpu_gated import DT, HF, SMALL, _api
from test_gpu_gated_forms import BWD_FORMS, FWD_FORMS

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "fp16"]


def zeros(N, K, dtype):
    q = _api()
    w = [q.qlora_nf4_quantize(torch.zeros(N, K, device=dev()), compute_dtype=dtype)
         for _ in range(2)]
    assert not q.qlora_nf4_dequantize(w[0]).any()
    return w


def check_fwd(T, N, K, r, dtype, s, **powers):
    """P of both projections."""
    q, dt = _api(), DT[dtype]
    X, A, B = E.forward_case(T, N, K, r, 1, dev(), **powers)
    h, saved = q.qlora_gated_linear_fwd(*zeros(N, K, dtype), X.to(dt), A[0].to(dt), B[0].to(dt),
                                        A[1].to(dt), B[1].to(dt), s * r)
    for i, (ref, err) in enumerate(E.projections(X, A, B, s, dt)):
        E.check(saved[i], ref, err, ("P", i, T, N, K, r))
    return X, A, h, saved


def check_bwd(T, N, K, r, dtype, s, **powers):
    q, dt = _api(), DT[dtype]
    dH, A, B, P = E.backward_case(T, N, K, r, 2, dev(), **powers)
    g = torch.Generator(device=dev()).manual_seed(3)
    X = E.pairs(g, K, T, dev()).T.contiguous().to(dt)
    U = [torch.randn(T, r, generator=g, device=dev()).to(dt) for _ in range(2)]
    got = q.qlora_gated_linear_bwd(*zeros(N, K, dtype), X, dH.to(dt), A[0].to(dt), B[0].to(dt),
                                   A[1].to(dt), B[1].to(dt), s * r,
                                   q.GatedSaved(P[0].to(dt), P[1].to(dt), *U))
    E.check(got[0], *E.dx(dH, A, B, P, s, dt), ("dX", T, N, K, r))
    for y, (ref, err) in zip(got[1::2], E.da(dH, X.double(), B, P, s, dt)):
        E.check(y, ref, err, ("dA", T, N, K, r))
    return dH, A, B, P, X, got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K,r", SMALL + FWD_FORMS)
def test_forward_keeps_two_terms(T, N, K, r, dtype):
    print(f"[gated] P {T} x {N} x {K} r {r} {dtype}", flush=True)
    check_fwd(T, N, K, r, dtype, 2.0 ** -6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K,r", SMALL + BWD_FORMS)
def test_dx_and_da_keep_their_terms(T, N, K, r, dtype):
    """|G| past 65504 at every size."""
    print(f"[gated] dX {T} x {N} x {K} r {r} {dtype}", flush=True)
    dH, _, B, P, _, _ = check_bwd(T, N, K, r, dtype, 2.0 ** -12)
    assert ((dH * P[0]) @ B[1]).abs().max() > 65504


# streaming, 128- and 256-row tiles whole and split, weights dequantised once
RANGES = [(3, 272, 1024, 32), (48, 272, 1024, 32), (64, 272, 1024, 32), (65, 272, 1024, 64),
          (300, 528, 1088, 64), (600, 1040, 448, 128), (2861, 2864, 1024, 16)]


@pytest.mark.parametrize("T,N,K,r", RANGES)
def test_forward_where_s_u_passes_the_largest_fp16_number(T, N, K, r):
    """s = 64, |s U| past 65504 and |U| below: P, H and U_save are finite, on both
    sides of the streaming form's border."""
    X, A, h, saved = check_fwd(T, N, K, r, "fp16", 64.0, a=2.0 ** -6, b=2.0 ** -14)
    u = (X @ A[0].T).abs().max()
    assert u < 65504 < 64 * u
    assert h.isfinite().all() and all(t.isfinite().all() for t in saved)


@pytest.mark.parametrize("T,N,K,r", RANGES)
def test_forward_where_u_passes_the_largest_fp16_number(T, N, K, r):
    """|U| past 65504: U_save is infinite there, P and H are right."""
    X, A, h, saved = check_fwd(T, N, K, r, "fp16", 2.0 ** -13)
    over = (X @ A[0].T).abs() >= 65520
    assert over.any() and torch.equal(saved.U_gate.isinf(), over)
    assert h.isfinite().all()


@pytest.mark.parametrize("T,N,K,r", RANGES)
def test_forward_of_small_values(T, N, K, r):
    """U near 2^-15, below fp16's normal numbers."""
    check_fwd(T, N, K, r, "fp16", 2.0 ** 8, x=2.0 ** -18, a=2.0 ** -14)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K,r", RANGES)
@pytest.mark.parametrize("s,powers", [(1.0, dict(a=2.0 ** -12)),
                                      (2.0 ** 6, dict(d=2.0 ** -24, b=2.0 ** -14, a=2.0 ** 6))],
                         ids=["large", "small"])
def test_gradients_of_any_size(T, N, K, r, s, powers, dtype):
    """s |G| past 65504; G near 2^-15, from dH below 2^-16."""
    print(f"[gated] dX {T} x {N} x {K} r {r} {dtype} {powers}", flush=True)
    dH, A, B, P, X, got = check_bwd(T, N, K, r, dtype, s, **powers)
    G = (dH * P[0]) @ B[1]
    assert got[0].isfinite().all()
    assert G.abs().max() > 65504 if s == 1.0 else G.abs().max() < 2.0 ** -10


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K,r", [(16, 272, 64, 16), (48, 272, 320, 48), (300, 144, 512, 64),
                                     (112, 400, 128, 112), (700, 256, 192, 128)])
def test_adapter_gradients_keep_every_term_of_d(T, N, K, r, dtype):
    """dA and dB pick single values of d out: bf16's third term and fp16's second."""
    q, dt = _api(), DT[dtype]
    dH, P, U, B, X, d = E.picked_case(T, N, K, r, 4, dev(), dt)
    A = torch.zeros(r, K, dtype=dt, device=dev())
    to = lambda *v: [t.to(dt) for t in v]  # noqa: E731
    dH, X, B, U = to(dH, X, B, U)
    got = q.qlora_gated_linear_bwd(*zeros(N, K, dtype), X, dH, A, B, A, B, 0.25 * r,
                                   q.GatedSaved(*to(*P), U, U))
    for i, ((dA, eA), (dB, eB)) in enumerate(E.picked(d, r, K, dt)):
        E.check(4.0 * got[1 + 2 * i], dA, eA, ("dA", i))
        E.check(4.0 * got[2 + 2 * i], dB, eB, ("dB", i))


def test_rows_far_apart_keep_their_bits():
    """128-row tiles 2^18 apart, and the rows of the two projections 2^10 and 2^18."""
    T, N, K, r = 400, 272, 512, 32
    q = _api()
    X, A, B = E.forward_case(T, N, K, r, 5, dev(), b=2.0 ** -10)
    X[:128] *= 2.0 ** -10
    X[256:384] *= 2.0 ** 8
    A[1] = A[1] * 2.0 ** -10
    to = lambda *v: [t.to(HF) for t in v]  # noqa: E731
    w = zeros(N, K, "fp16")
    _, saved = q.qlora_gated_linear_fwd(*w, *to(X, A[0], B[0], A[1], B[1]), r / 16)
    for i, (ref, err) in enumerate(E.projections(X, A, B, 1 / 16, HF)):
        E.check(saved[i], ref, err, ("P", i))
    dH, A, B, P = E.backward_case(T, N, K, r, 6, dev(), up=2.0 ** -12)
    dH[:128] *= 2.0 ** -14
    dH[256:384] *= 2.0 ** 3
    U = [torch.zeros(T, r, dtype=HF, device=dev()) for _ in range(2)]
    got = q.qlora_gated_linear_bwd(*w, *to(X, dH, A[0], B[0], A[1], B[1]), 2.0 ** -14 * r,
                                   q.GatedSaved(*to(*P), *U))
    E.check(got[0], *E.dx(dH, A, B, P, 2.0 ** -14, HF), "dX")
    X = E.pairs(torch.Generator(device=dev()).manual_seed(9), K, T, dev()).T.contiguous()
    got = q.qlora_gated_linear_bwd(*w, *to(X, dH, A[0], B[0], A[1], B[1]), 2.0 ** -14 * r,
                                   q.GatedSaved(*to(*P), *U))
    for y, (ref, err) in zip(got[1::2], E.da(dH, X, B, P, 2.0 ** -14, HF)):
        E.check(y, ref, err, "dA")


def test_fp16_scales_are_formed_anew_in_every_replay():
    q = _api()
    T, N, K, r = 300, 272, 512, 48
    X, A, B = E.forward_case(T, N, K, r, 7, dev())
    dH, _, _, P = E.backward_case(T, N, K, r, 8, dev())
    w = zeros(N, K, "fp16")
    adapters = [t.to(HF) for t in (A[0], B[0], A[1], B[1])]
    U = [torch.ones(T, r, dtype=HF, device=dev()) for _ in range(2)]
    kept = q.GatedSaved(P[0].to(HF), P[1].to(HF), *U)
    alpha = 2.0 ** -14 * r

    def run(x, dh):
        h, s = q.qlora_gated_linear_fwd(*w, x, *adapters, alpha)
        return [h, *s, *q.qlora_gated_linear_bwd(*w, x, dh, *adapters, alpha, kept)]

    inputs = [[(X * 2.0 ** p).to(HF), (dH * 2.0 ** p).to(HF)] for p in (0, -12, 2)]
    ref = [run(*i) for i in inputs]
    live = [t.clone() for t in inputs[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*live)
    for k in (0, 2, 1, 2, 0, 1):
        for s, t in zip(live, inputs[k]):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref[k])), k
        run(*inputs[1])
        torch.cuda.synchronize()

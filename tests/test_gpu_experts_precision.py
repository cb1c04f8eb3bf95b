"""How much of U and G = dY B the expert-grouped layer keeps, against the 64-bit
formulas with bounds per element that leave no room for one 16-bit rounding."""
import numpy as np
import pytest
import torch

from experts_ref import U_ACC, grouped_backward, grouped_forward, group_bounds
from gpu_util import dev
from test_gpu_experts import ALPHA, BF, HALF, HF, backward, forward, host, make, within

pytestmark = pytest.mark.gpu


def check_da(c, dtype, r):
    """dA of every expert within float32 sums of 22 bits of G.  In fp16 a G far
    below the largest of its rows is off by 2^-39 of the bound that the scale of
    its terms is taken from: at most 2 S max |partial| with S <= 128 parts, each
    at most |dY_t| |B_p| (Cauchy-Schwarz): 2^-31 of the largest of those."""
    U = forward(c)[1]
    _, dA, _ = backward(c, U)
    x, dy, a, b, u = (host(t) for t in (c["X"], c["dY"], c["A"], c["B"], U))
    _, da, _ = grouped_backward(x, dy, c["W"], a, b, c["off"], ALPHA, u)
    for e in range(len(c["off"]) - 1):
        i, j = c["off"][e], c["off"][e + 1]
        lim = group_bounds(x[i:j], dy[i:j], c["W"][e], a[e], b[e], ALPHA, HALF[dtype])["da"]
        if j > i:
            top = np.sqrt((dy[i:j] ** 2).sum(1)).max() * np.sqrt((b[e] ** 2).sum(0)).max()
            lim = lim + ALPHA / r * 2.0 ** -31 * top * np.abs(x[i:j]).sum(0)
        got = host(dA[e])
        assert np.isfinite(got).all(), e
        within(("dA", e), got, da[e], lim)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("power", [-16, -12, -6])
def test_small_gradients(power, dtype):
    """dY of 2^power with a young B: G lies far below fp16's normal range."""
    c = make([90, 0, 200, 131, 7], 272, 576, 32, dtype, seed=power)
    c["dY"] = (c["dY"].float() * 2.0 ** power).to(dtype)
    c["B"] = (c["B"].float() * 0.125).to(dtype)
    check_da(c, dtype, 32)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_gradients_past_the_largest_fp16_number(dtype):
    """|G| past 2^16 in fp16: dA, which sums it in float32, is finite and exact."""
    c = make([90, 0, 200, 131, 7], 272, 576, 64, dtype, seed=9)
    c["dY"] = (c["dY"].float() * 512).to(dtype)
    c["B"] = (c["B"].float() * 800).to(dtype)
    c["A"] = (c["A"].float() * 0.125).to(dtype)
    assert np.abs(host(c["dY"][:90]) @ host(c["B"][0])).max() > 2.0 ** 17
    check_da(c, dtype, 64)


def test_one_large_row_leaves_the_others_their_bits():
    """Rows 2^20 apart in one expert, and experts that far apart: each keeps
    what its bound says."""
    c = make([90, 60, 200], 272, 576, 16, HF, seed=3)
    s = torch.ones(350, 1, device=dev())
    s[:90] = 2.0 ** -8
    s[150:] = 2.0 ** -10
    s[200] = 2.0 ** 10
    c["dY"] = (c["dY"].float() * s).to(HF)
    check_da(c, HF, 16)


def test_fp16_backward_in_a_graph():
    """The scale of G's terms is formed anew in every replay: rows that grow
    and shrink between replays give what the eager call gives."""
    c = make([90, 0, 200, 31], 272, 576, 16, HF, seed=5)
    U = forward(c)[1]
    dys = [(c["dY"].float() * 2.0 ** p).to(HF) for p in (0, -14, 8)]
    ref = []
    for dy in dys:
        c["dY"] = dy
        ref.append(backward(c, U))
    torch.cuda.synchronize()
    c["dY"] = dys[0].clone()
    out = [torch.empty_like(t) for t in ref[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        backward(c, U, dX=out[0], dA=out[1], dB=out[2])
    live = c["dY"]
    for i in (0, 2, 1, 2, 0, 1):
        live.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref[i], out)), i
        c["dY"] = dys[1]
        backward(c, U)
        torch.cuda.synchronize()


# --------------------------------------------------------------------------
# U and G on their way to Y and dX
# --------------------------------------------------------------------------
def two_term_bounds(x, dy, w, a, b, half, dtype, r):
    """Bounds per element of one expert's Y and dX where s U and G meet B and A as
    two 16-bit terms, half^2 of them relative to the value; float32 sums (over K
    or N, then over both terms' r columns) as in group_bounds; s U is one more
    product in float32 (2^-24), as are s and the scale of the terms of G; the
    output's rounding.  fp16: a term of s U is no closer than 2^-25 (half the
    smallest number; not s times that), one of G than 2^-31 of the largest |dY_t|
    |B_p| (see check_da), an output no closer than 2^-25."""
    s = ALPHA / r
    n = lambda m, ax: np.sqrt((m * m).sum(ax))  # noqa: E731
    K, N = x.shape[1], w.shape[0]
    u, g = x @ a.T, dy @ b
    y, dx = x @ w.T + s * (u @ b.T), dy @ w + s * (g @ a)
    eu = s * ((half ** 2 + 2.0 ** -24) * np.abs(u) + 1.01 * K * U_ACC * np.outer(n(x, 1), n(a, 1)))
    eg = half ** 2 * np.abs(g) + 1.01 * N * U_ACC * np.outer(n(dy, 1), n(b, 0))
    tiny = 0.0
    if dtype == HF:
        tiny = 2.0 ** -25
        eu = eu + tiny
        eg = eg + 2.0 ** -31 * n(dy, 1).max() * n(b, 0).max()
    ly = (1.01 * (K + 2 * r + 4) * U_ACC * (np.outer(n(x, 1), n(w, 1)) + s * np.outer(n(u, 1), n(b, 1)))
          + 1.01 * eu @ np.abs(b).T + half * np.abs(y) + tiny)
    ldx = (1.01 * (N + 2 * r + 4) * U_ACC * (np.outer(n(dy, 1), n(w, 0)) + s * np.outer(n(g, 1), n(a, 0)))
           + 1.01 * s * eg @ np.abs(a) + half * np.abs(dx) + tiny)
    return ly, ldx


def check_outputs(c, dtype, r):
    Y, U = forward(c)
    dX = backward(c, U)[0]
    x, dy, a, b, u = (host(t) for t in (c["X"], c["dY"], c["A"], c["B"], U))
    y, _ = grouped_forward(x, c["W"], a, b, c["off"], ALPHA)
    dx = grouped_backward(x, dy, c["W"], a, b, c["off"], ALPHA, u)[0]
    assert Y.isfinite().all() and dX.isfinite().all()
    for e in range(len(c["off"]) - 1):
        i, j = c["off"][e], c["off"][e + 1]
        if j > i:
            ly, ldx = two_term_bounds(x[i:j], dy[i:j], c["W"][e], a[e], b[e], HALF[dtype], dtype, r)
            within(("Y", e), host(Y[i:j]), y[i:j], ly)
            within(("dX", e), host(dX[i:j]), dx[i:j], ldx)


FORMS = {"stream_16": [5, 0, 3, 9], "stream_32": [20, 0, 33, 9], "tiles_128": [90, 0, 200, 131, 7],
         "split_tiles": [130, 300, 257], "tiles_256": [300, 0, 129] + [257] * 22}
SHAPES = {"tiles_256": (1040, 1088)}      # N, K; else 272, 576


@pytest.mark.parametrize("r", [16, 48, 64, 112, 128])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("form", list(FORMS))
def test_adapters_cost_no_more_than_the_output_rounding(form, dtype, r):
    N, K = SHAPES.get(form, (272, 576))
    c = make(FORMS[form], N, K, r, dtype, seed=r)
    c["B"] = (c["B"].float() * 4).to(dtype)      # a trained B: s U B as large as X W
    check_outputs(c, dtype, r)


@pytest.mark.parametrize("form", ["tiles_128", "tiles_256"])
@pytest.mark.parametrize("power", [-14, 5])
def test_gradients_of_any_size_reach_dx(form, power):
    N, K = SHAPES.get(form, (272, 576))
    c = make(FORMS[form], N, K, 32, HF, seed=power)
    c["dY"] = (c["dY"].float() * 2.0 ** power).to(HF)
    check_outputs(c, HF, 32)


def test_dx_where_s_g_passes_the_largest_fp16_number():
    """The same values as above: s |G| passes 65504, dX does not."""
    c = make([90, 0, 200, 131, 7], 272, 576, 64, HF, seed=9)
    c["dY"] = (c["dY"].float() * 512).to(HF)
    c["B"] = (c["B"].float() * 800).to(HF)
    c["A"] = (c["A"].float() * 0.125).to(HF)
    dX, dA, _ = backward(c, forward(c)[1])
    g = np.abs(host(c["dY"][:90]) @ host(c["B"][0]))
    assert g.max() > 2.0 ** 18 and dX.isfinite().all() and dA.isfinite().all()


def test_values_past_fp16_stay_infinite():
    """U past 65504: U_save and Y are infinite, as one 16-bit U gives, not NaN."""
    c = make([5, 3], 64, 128, 16, HF, seed=2)
    for counts in ([5, 3], [90, 200]):
        c = make(counts, 64, 128, 16, HF, seed=2)
        c["A"][:] = 0
        c["A"][:, 0] = 600.0
        c["X"] = c["X"].abs() + 1
        c["B"][:] = 0
        c["B"][:, :, 0] = 0.01
        Y, U = forward(c)
        assert (U[:, 0] == float("inf")).all() and (Y == float("inf")).all()


@pytest.mark.parametrize("form", ["stream_16", "stream_32", "tiles_128", "tiles_256"])
def test_y_where_u_passes_the_largest_fp16_number(form):
    """|U| past 65504 with s = 1/4: U_save is infinite there, but s U and Y are
    finite, and right."""
    N, K = SHAPES.get(form, (272, 576))
    c = make(FORMS[form], N, K, 64, HF, seed=11)
    c["A"] = (c["A"].float() * 10000).to(HF)
    c["B"] = (c["B"].float() * 0.125).to(HF)
    Y, U = forward(c)
    x, a, b = (host(c[k]) for k in ("X", "A", "B"))
    y, u = grouped_forward(x, c["W"], a, b, c["off"], ALPHA)
    assert np.abs(u).max() > 1.2 * 65504 and 0.25 * np.abs(u).max() < 65504
    assert U.isinf().any() and Y.isfinite().all()
    for e in range(len(c["off"]) - 1):
        i, j = c["off"][e], c["off"][e + 1]
        if j > i:
            dy = np.zeros((j - i, N))
            ly, _ = two_term_bounds(x[i:j], dy, c["W"][e], a[e], b[e], HALF[HF], HF, 64)
            within(("Y", e), host(Y[i:j]), y[i:j], ly)

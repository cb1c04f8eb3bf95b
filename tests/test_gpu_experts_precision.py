"""How much of U and G = dY B the expert-grouped layer keeps, against the 64-bit
formulas with bounds per element that leave no room for one 16-bit rounding."""
import numpy as np
import pytest
import torch

from experts_ref import grouped_backward, group_bounds
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

"""A training step of the expert-grouped layer against differences of its loss
in the 64-bit formulas."""
import numpy as np
import pytest
import torch

from experts_ref import U_ACC, db_bound, grouped_forward, group_bounds
from gpu_util import dev
from test_gpu_experts import ALPHA, BF, HALF, HF, _api, backward, forward, host, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[5, 0, 3, 9], [40, 0, 125, 90]], ids=["stream", "tiles"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_a_step_changes_the_loss_by_what_the_gradients_say(counts, dtype):
    """Loss sum(Y dY).  Y is bilinear in A and B, so a step (a, b) changes it by
    exactly <gA, a> + <gB, b> + s sum(dY (X a^T) b^T) with the true gradients.
    With the kernel's in their place the two sides differ by at most their
    bounds times |a| and |b|; gB's also by the rounding of the saved U."""
    q = _api()
    r, lr = 16, 1e-3
    c = make(counts, 144, 320, r, dtype, lead=2, tail=1, seed=4, junk=0.0)
    _, U = forward(c)
    _, dA, dB = backward(c, U)
    step = {}
    for name, grad in (("A", dA), ("B", dB)):
        p = c[name].float()
        before = p.clone()
        q.qlora_adamw_step(p, torch.zeros_like(p), torch.zeros_like(p), grad, 1, lr)
        step[name] = host(p) - host(before)
    x, dy, A, B, u = (host(t) for t in (c["X"], c["dY"], c["A"], c["B"], U))
    off, s = c["off"], ALPHA / r

    def loss(a, b):
        return (grouped_forward(x, c["W"], a, b, off, ALPHA)[0] * dy).sum()

    change = loss(A + step["A"], B + step["B"]) - loss(A, B)
    said, room, size = 0.0, 0.0, 0.0
    for e in range(len(counts)):
        i, j = off[e], off[e + 1]
        xe, dye, a, b = x[i:j], dy[i:j], step["A"][e], step["B"][e]
        said += (host(dA[e]) * a).sum() + (host(dB[e]) * b).sum()
        said += s * (dye * ((xe @ a.T) @ b.T)).sum()
        size += np.abs(s * dye * ((xe @ a.T) @ b.T)).sum() + np.abs(host(dA[e]) * a).sum()
        if j > i:
            lim = group_bounds(xe, dye, c["W"][e], A[e], B[e], ALPHA, HALF[dtype])
            tiny = 2.0 ** -25 if dtype == HF else 0.0
            top = np.sqrt((dye ** 2).sum(1)).max() * np.sqrt((B[e] ** 2).sum(0)).max()
            da = lim["da"] + (s * 2.0 ** -31 * top * np.abs(xe).sum(0) if tiny else 0.0)
            db = db_bound(dye, u[i:j], ALPHA, r) + s * np.abs(dye).T @ (lim["u"] + tiny)
            room += (da * np.abs(a)).sum() + (db * np.abs(b)).sum()
    # the 64-bit sums themselves
    room += 1e-12 * (np.abs(loss(A, B)) + size + np.abs(grouped_forward(x, c["W"], A, B, off, ALPHA)[0] * dy).sum())
    assert not step["A"][1].any() and not step["B"][1].any()     # the expert without rows
    assert abs(change - said) <= room, (change, said, room)
    # a step against the gradients lowers the loss by far more than that room
    assert change < -4 * room, (change, room)

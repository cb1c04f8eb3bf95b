"""Calls of the expert-grouped and the 8-bit layer that the documentation allows:
several at once, odd offsets, a workspace of exactly its size and the longest
batches, with the fp16 backward's scales among what they share."""
import numpy as np
import pytest
import torch

from experts_ref import db_bound, grouped_backward, group_bounds
from gpu_util import dev
from test_gpu_experts import ALPHA, BF, HALF, HF, _api, backward, check, forward, host, make, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [129], [128, 1, 127]],
                         ids=["one", "one_of_three", "129", "borders_of_128"])
def test_smallest_groups(counts, dtype):
    check(make(counts, 32, 64, 16, dtype, 1, 1), dtype, 16)


def test_offsets_out_of_range_in_fp16():
    c = make([100, 160, 40], 272, 576, 16, HF)
    Y, U = forward(c)
    g = backward(c, U)
    c["offsets"] = torch.tensor([-5, 100, 260, 1 << 30], dtype=torch.int32, device=dev())
    Y2, U2 = forward(c)
    assert torch.equal(Y, Y2) and torch.equal(U, U2)
    assert all(torch.equal(a, b) for a, b in zip(g, backward(c, U)))


@pytest.mark.parametrize("off", [[0, 150, 20, 200], [200, 0, 300, -7], [7, 7, 3, 3],
                                 [1 << 30, -9, 200, 0]])
def test_offsets_that_decrease_in_fp16_stay_inside_the_workspace(off):
    """Outputs are unspecified; nothing behind the workspace or the outputs is
    written."""
    q = _api()
    c = make([100, 60, 40], 272, 576, 16, HF)
    c["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev())
    n = q.qlora_grouped_linear_workspace(200, 3, 272, 576, 16, "fp16", True)
    buf = torch.zeros(n + 8192, dtype=torch.uint8, device=dev())
    buf[n:] = 0x5A
    U = torch.zeros(200, 16, dtype=HF, device=dev())
    outs = []
    for t in (torch.Size([200, 576]), c["A"].shape, c["B"].shape):
        k = int(np.prod(t))
        flat = torch.full((k + 4096,), 5.0, dtype=HF if not outs else torch.float32, device=dev())
        outs.append((flat, k, t))
    dX, dA, dB = (f[:k].view(t) for f, k, t in outs)
    backward(c, U, dX=dX, dA=dA, dB=dB, workspace=buf[:n])
    assert (buf[n:] == 0x5A).all()
    for f, k, _ in outs:
        assert (f[k:] == 5).all()


@pytest.mark.parametrize("counts,N,K,r", [([2, 0, 1, 3], 272, 576, 16), ([90, 0, 200, 31], 272, 576, 48),
                                          ([130, 300, 257], 2080, 1088, 64)],
                         ids=["few", "tiles", "split_tiles"])
def test_workspace_of_exactly_its_size_in_fp16(counts, N, K, r):
    q = _api()
    c = make(counts, N, K, r, HF)
    T, E = c["T"], len(counts)
    ref = forward(c)
    gref = backward(c, ref[1])
    for bwd in (False, True):
        n = q.qlora_grouped_linear_workspace(T, E, N, K, r, "fp16", bwd)
        buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=dev())
        for _ in range(3):
            out = backward(c, ref[1], workspace=buf[:n]) if bwd else forward(c, workspace=buf[:n])
            assert all(torch.equal(a, b) for a, b in zip(out, gref if bwd else ref))
        assert (buf[n:] == 0xFF).all()


def _on(stream, f):
    with torch.cuda.stream(stream):
        return f()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_two_streams_at_once(dtype):
    """Two layers' calls interleaved on two streams, each with workspaces of its
    own, give what they give one after the other."""
    q = _api()
    cs = [make([130, 0, 257, 31], 528, 1088, 32, dtype, seed=s) for s in (1, 2)]
    xs = [torch.randn(150 + s, 1040, device=dev()).to(dtype) for s in (1, 2)]
    ws = [q.Int8Weight(*q.qlora_int8_quantize(torch.randn(272, 1040, device=dev()))) for _ in xs]

    def all_of(i):
        Y, U = forward(cs[i])
        return (Y, U) + tuple(backward(cs[i], U)) + (q.qlora_int8_linear_fwd(ws[i], xs[i]),)

    ref = [all_of(i) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i in (0, 1):
            got[i].append(_on(streams[i], lambda: all_of(i)))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, ref[i]))


def test_two_graphs_replayed_at_once():
    """Graphs captured one after the other, each with buffers and a workspace of
    its own, replayed on two streams."""
    q = _api()
    cs = [make([130, 0, 257, 31], 528, 1088, 32, HF, seed=s) for s in (3, 4)]
    ref, outs, graphs = [], [], []
    for c in cs:
        Y, U = forward(c)
        ref.append((Y, U) + tuple(backward(c, U)))
        outs.append([torch.empty_like(t) for t in ref[-1]])
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        n = [q.qlora_grouped_linear_workspace(c["T"], 4, 528, 1088, 32, "fp16", b) for b in (0, 1)]
        w = [torch.empty(v, dtype=torch.uint8, device=dev()) for v in n]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            forward(c, Y=o[0], U_save=o[1], workspace=w[0])
            backward(c, o[1], dX=o[2], dA=o[3], dB=o[4], workspace=w[1])
        graphs.append((g, w))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(5):
        for o in outs:
            for t in o:
                t.fill_(3)
        torch.cuda.synchronize()
        for s, (g, _) in zip(streams, graphs):
            _on(s, g.replay)
        torch.cuda.synchronize()
        for o, want in zip(outs, ref):
            assert all(torch.equal(a, b) for a, b in zip(o, want)), k
        forward(cs[0])
        torch.cuda.synchronize()


def test_long_batch_in_fp16():
    """A million rows, byte offsets past 2^31, gradients of 2^-14: 7814 tiles'
    scales, most of rows that hold only zeros."""
    T, N, K, r = 1_000_000, 16, 1024, 16
    q = _api()
    g = torch.Generator(device=dev()).manual_seed(1)
    w = q.qlora_nf4_quantize(torch.randn(2 * N, K, generator=g, device=dev()) * 0.02,
                             compute_dtype="fp16")
    X = torch.zeros(T, K, dtype=HF, device=dev())
    rows = [0, 1, 127, 128, 499_999, 500_000, T - 200, T - 1]
    X[rows] = torch.randn(len(rows), K, generator=g, device=dev()).to(HF)
    A = (torch.randn(2, r, K, generator=g, device=dev()) / 4).to(HF)
    B = (torch.randn(2, N, r, generator=g, device=dev()) * 0.01).to(HF)
    off = [0, 500_000, T]
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    _, U = q.qlora_grouped_linear_fwd(w, X, offsets, A, B, ALPHA)
    W = q.qlora_nf4_dequantize(w).double().view(2, N, K).cpu().numpy()
    dY = torch.zeros(T, N, dtype=HF, device=dev())
    dY[rows] = (torch.randn(len(rows), N, generator=g, device=dev()) * 2.0 ** -14).to(HF)
    dX, dA, dB = q.qlora_grouped_linear_bwd(w, X, dY, offsets, A, B, ALPHA, U)
    sel = torch.tensor(rows, device=dev())
    small = [0, sum(t < off[1] for t in rows), len(rows)]
    x, dy, u, a, b = host(X[sel]), host(dY[sel]), host(U[sel]), host(A), host(B)
    dx_ref, da_ref, db_ref = grouped_backward(x, dy, W, a, b, small, ALPHA, u)
    for e in range(2):
        i, j = small[e], small[e + 1]
        lim = group_bounds(x[i:j], dy[i:j], W[e], a[e], b[e], ALPHA, HALF[HF])
        top = np.sqrt((dy[i:j] ** 2).sum(1)).max() * np.sqrt((b[e] ** 2).sum(0)).max()
        floor = ALPHA / r * 2.0 ** -31 * top
        within("dX", host(dX[sel])[i:j], dx_ref[i:j],
               lim["dx"] + 2.0 ** -25 + floor * np.abs(a[e]).sum(0))
        within("dA", host(dA[e]), da_ref[e], lim["da"] + floor * np.abs(x[i:j]).sum(0))
        within("dB", host(dB[e]), db_ref[e], db_bound(dy[i:j], u[i:j], ALPHA, r))
    dX[sel] = 0
    assert not dX.any()

"""The expert-grouped linear layer on the GPU, expert by expert against the
64-bit formulas with bounds per element."""
import numpy as np
import pytest
import torch

from experts_ref import db_bound, grouped_backward, grouped_forward, group_bounds
from gpu_util import dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11}
ALPHA = 16.0


def _api():
    import bit_nf4_quantized_06_amd as q
    return q


def make(counts, N, K, r, dtype, lead=0, tail=0, dq=True, seed=0, junk=float("nan")):
    """A stacked weight, adapters, rows; `lead` and `tail` rows belong to no
    expert and hold `junk`."""
    q = _api()
    g = torch.Generator(device=dev()).manual_seed(seed)
    E, T = len(counts), sum(counts) + lead + tail
    rnd = lambda *n: torch.randn(*n, generator=g, device=dev())  # noqa: E731
    c = {"off": [lead + int(v) for v in np.concatenate([[0], np.cumsum(counts)])], "T": T}
    c["offsets"] = torch.tensor(c["off"], dtype=torch.int32, device=dev())
    c["w"] = q.qlora_nf4_quantize(rnd(E * N, K) * 0.02, double_quant=dq,
                                  compute_dtype="fp16" if dtype == HF else "bf16")
    c["X"], c["dY"] = rnd(T, K).to(dtype), rnd(T, N).to(dtype)
    for t in (c["X"], c["dY"]):
        t[:lead] = junk
        t[T - tail:] = junk
    c["A"], c["B"] = (rnd(E, r, K) / r ** 0.5).to(dtype), (rnd(E, N, r) * 0.01).to(dtype)
    c["W"] = q.qlora_nf4_dequantize(c["w"]).double().cpu().numpy().reshape(E, N, K)
    return c


def forward(c, **kw):
    return _api().qlora_grouped_linear_fwd(c["w"], c["X"], c["offsets"], c["A"], c["B"], ALPHA,
                                           **kw)


def backward(c, U, **kw):
    return _api().qlora_grouped_linear_bwd(c["w"], c["X"], c["dY"], c["offsets"], c["A"], c["B"],
                                           ALPHA, U, **kw)


def host(t):
    return t.double().cpu().numpy()


def within(what, got, ref, lim):
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           got[bad][:4], ref[bad][:4], lim[bad][:4])


def check(c, dtype, r, run_bwd=True):
    T, N, K = c["T"], c["W"].shape[1], c["W"].shape[2]
    off = c["off"]
    Y = torch.full((T, N), 7.0, dtype=dtype, device=dev())
    U = torch.full((T, r), 7.0, dtype=dtype, device=dev())
    forward(c, Y=Y, U_save=U)
    x, dy, a, b, u = (host(c[k]) if k in c else host(U) for k in ("X", "dY", "A", "B", "U"))
    inside = slice(off[0], off[-1])
    xz, dyz, uz = np.zeros(x.shape), np.zeros(dy.shape), np.zeros(u.shape)
    xz[inside], dyz[inside], uz[inside] = x[inside], dy[inside], u[inside]
    y_ref, u_ref = grouped_forward(xz, c["W"], a, b, off, ALPHA)
    outs = [("Y", Y), ("U", U)]
    if run_bwd:
        dX = torch.full((T, K), 7.0, dtype=dtype, device=dev())
        dA = torch.full(c["A"].shape, 7.0, device=dev())
        dB = torch.full(c["B"].shape, 7.0, device=dev())
        backward(c, U, dX=dX, dA=dA, dB=dB)
        outs.append(("dX", dX))
        dx_ref, da_ref, db_ref = grouped_backward(xz, dyz, c["W"], a, b, off, ALPHA, uz)
    for name, t in outs:
        assert (t[:off[0]] == 7).all() and (t[off[-1]:] == 7).all(), f"{name}: rows of no expert"
    for e in range(len(off) - 1):
        i, j = off[e], off[e + 1]
        lim = group_bounds(xz[i:j], dyz[i:j], c["W"][e], a[e], b[e], ALPHA, HALF[dtype])
        # fp16 below its normal range rounds to steps of 2^-24
        tiny = 2.0 ** -25 if dtype == HF else 0.0
        within(("Y", e), host(Y[i:j]), y_ref[i:j], lim["y"] + tiny)
        within(("U", e), host(U[i:j]), u_ref[i:j], lim["u"] + tiny)
        if run_bwd:
            within(("dX", e), host(dX[i:j]), dx_ref[i:j], lim["dx"] + tiny)
            # a term of G below fp16's normal range is off by 2^-25 at most
            g_tiny = tiny * ALPHA / r * np.abs(xz[i:j]).sum(0)
            within(("dA", e), host(dA[e]), da_ref[e], lim["da"] + g_tiny)
            within(("dB", e), host(dB[e]), db_ref[e], db_bound(dyz[i:j], uz[i:j], ALPHA, r))


WIDE = [200, 0, 513, 257, 100, 129, 256, 30, 70, 300, 128, 3]

# counts of rows per expert, N, K, r, type, rows before and behind, double quantisation
CASES = [
    ("one_row", [1], 64, 64, 16, BF, 0, 0, True),
    ("single_tile_rows", [5, 0, 3], 48, 128, 16, BF, 2, 3, True),
    ("no_rows", [0, 0], 32, 64, 16, BF, 0, 4, True),
    ("first_and_last_empty", [0, 9, 0], 32, 64, 16, HF, 0, 0, True),
    ("few_of_many", [1, 1, 0, 0, 2, 0, 0, 1], 1040, 2048, 16, HF, 0, 0, True),
    ("stream_tiles_16", [17, 0, 3, 1, 0, 0, 5, 2], 272, 576, 32, BF, 1, 1, True),
    ("stream_tiles_32", [33, 0, 10, 9], 272, 576, 32, BF, 1, 1, False),
    ("stream_tiles_64", [20, 0, 130, 65], 272, 576, 32, HF, 1, 1, True),
    ("stream_past_64_rows", [64, 100, 0, 65, 33, 97], 528, 1088, 48, BF, 3, 2, True),
    ("stream_one_expert", [63], 1040, 4096, 16, HF, 0, 0, False),
    ("tiles_few_rows", [24, 25, 0, 60, 9, 31, 2, 40, 70, 1], 5008, 1408, 16, BF, 2, 0, True),
    ("tiles_ragged", [300, 0, 70, 9], 272, 576, 48, HF, 1, 1, True),
    ("tiles_borders", [256, 257, 255, 1, 511], 528, 1088, 64, BF, 0, 5, False),
    ("rank_128", [700, 257], 272, 1024, 128, BF, 3, 0, True),
    ("rank_112", [130, 257, 0], 272, 1024, 112, HF, 3, 0, True),
    ("rank_80", [3] * 70, 144, 320, 80, BF, 0, 0, True),
    ("past_64_experts", [100] * 70 + [0] * 3, 80, 192, 16, HF, 0, 2, True),
    ("one_takes_all", [0, 1500, 0, 0], 272, 1088, 16, BF, 0, 0, True),
    # rows and columns that leave partial tiles in both directions, blocks of
    # an expert that start inside a group of 256
    ("partial_tiles", [200, 0, 40, 64, 65, 500], 1008, 512, 16, BF, 0, 7, False),
    # more tiles than the chip holds at a time, the last round's split in two,
    # with tiles of 128 and of 256 rows
    ("rounds_of_128", [130] * 37, 2080, 576, 16, BF, 0, 0, True),
    ("rounds_of_256", [300] * 20, 2080, 576, 16, HF, 0, 0, True),
    ("most_experts", [0, 1, 0, 2] * 256, 16, 64, 16, BF, 1, 0, True),
    ("most_experts_tiles", [70] * 1023 + [3], 16, 64, 16, HF, 0, 1, True),
    # 256-row tiles (more than 160 rows an expert and more than 96 tiles): halves
    # without rows, borders, empty experts, split tiles, every format and rank
    ("wide_tiles", WIDE, 2064, 2112, 48, BF, 1, 2, True),
    ("wide_tiles_fp16_constants", WIDE, 2064, 2112, 112, HF, 0, 3, False),
    ("wide_tiles_rank_128", WIDE, 2064, 2112, 128, BF, 3, 0, False),
    ("wide_tiles_one_expert", [2900], 2320, 2368, 16, BF, 0, 5, True),
    ("wide_reduction", [90, 170], 16, 11008, 32, HF, 0, 0, True),
    ("long_backward_reduction", [90, 170], 5520, 64, 32, BF, 0, 0, True),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_against_formulas(case):
    name, counts, N, K, r, dtype, lead, tail, dq = case
    print(f"[experts] {name}", flush=True)
    check(make(counts, N, K, r, dtype, lead, tail, dq), dtype, r)


def test_rows_of_no_expert_do_not_reach_the_others():
    """Infinities and NaN in rows that belong to no expert change nothing."""
    res = []
    for junk in (0.0, float("inf"), float("nan")):
        for counts in ([3, 2], [90, 170]):
            c = make(counts, 144, 320, 16, BF, 5, 9, junk=junk)
            Y, U = (torch.zeros(c["T"], n, dtype=BF, device=dev()) for n in (144, 16))
            forward(c, Y=Y, U_save=U)
            dX = torch.zeros(c["T"], 320, dtype=BF, device=dev())
            _, dA, dB = backward(c, U, dX=dX)
            res.append((Y, U, dX, dA, dB))
    for k in (2, 4):
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(res[i], res[k + i]))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts", [[5, 0, 3, 9], [90, 0, 200, 131], [300, 400, 257]],
                         ids=["stream", "tiles_128", "tiles_ragged"])
def test_values_that_are_not_finite_stay_with_their_row(counts, dtype, bad):
    """One such value in X reaches its row of Y and U, one in dY its row of dX,
    its expert's dA and its own row of that expert's dB; nothing else changes."""
    N, K, r, col = 272, 576, 16, 37
    c = make(counts, N, K, r, dtype)
    clean = forward(c)
    gclean = backward(c, clean[1])
    e = len(counts) - 1
    t = c["off"][e] + 1
    rest = torch.arange(c["T"], device=dev()) != t
    x = c["X"].clone()
    c["X"][t, col] = bad
    for got, ref in zip(forward(c), clean):
        assert torch.equal(got[rest], ref[rest]) and not got[t].isfinite().any()
    c["X"] = x
    c["dY"][t, col] = bad
    dX, dA, dB = backward(c, clean[1])
    assert torch.equal(dX[rest], gclean[0][rest]) and not dX[t].isfinite().any()
    assert torch.equal(dA[:e], gclean[1][:e]) and not dA[e].isfinite().any()
    assert torch.equal(dB[:e], gclean[2][:e]) and not dB[e, col].isfinite().any()
    others = torch.arange(N, device=dev()) != col
    assert torch.equal(dB[e][others], gclean[2][e][others])


def test_one_expert_is_the_dense_layer():
    """E = 1 over all rows against qlora_linear_fwd / _bwd: same weights, same
    formulas; both within their bounds of each other's."""
    q = _api()
    for T in (9, 40, 300):
        c = make([T], 272, 576, 32, BF)
        check(c, BF, 32)
        Y, U = forward(c)
        Yd, Ud = q.qlora_linear_fwd(c["w"], c["X"], c["A"][0], c["B"][0], ALPHA)
        n = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
        # two results within half a 16-bit step each (Y: two more from s U)
        assert n(Y, Yd) <= 4 * HALF[BF] and n(U, Ud) <= 2 * HALF[BF]


def test_deterministic_and_weight_untouched():
    c = make([300, 0, 70, 9], 272, 576, 48, BF)
    before = [t.clone() for t in (c["w"].codes, c["w"].absmax_code, c["w"].absmax_scale)]
    Y, U = forward(c)
    g = backward(c, U)
    for _ in range(3):
        Y2, U2 = forward(c)
        assert torch.equal(Y, Y2) and torch.equal(U, U2)
        assert all(torch.equal(a, b) for a, b in zip(g, backward(c, U)))
    assert all(torch.equal(a, b) for a, b in
               zip(before, (c["w"].codes, c["w"].absmax_code, c["w"].absmax_scale)))


def test_no_rows_at_all():
    c = make([4, 4], 32, 64, 16, BF)
    c["X"], c["dY"] = c["X"][:0], c["dY"][:0]
    c["offsets"] = torch.zeros(3, dtype=torch.int32, device=dev())
    Y, U = forward(c)
    assert Y.shape == (0, 32) and U.shape == (0, 16)
    dX, dA, dB = backward(c, U)
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()


def test_without_u():
    c = make([300, 70], 272, 576, 16, BF)
    Y, U = forward(c)
    Y2, none = forward(c, save_u=False)
    assert none is None and torch.equal(Y, Y2)


@pytest.mark.parametrize("counts", [[2, 0, 1, 3], [90, 0, 200, 31]], ids=["stream", "tiles"])
def test_streams_and_graph(counts):
    """On a caller's stream, and captured: the offsets are device data, so a
    replay follows new counts; each replay equals the eager call."""
    q = _api()
    c = make(counts, 272, 576, 16, BF)
    T, r = c["T"], 16
    offs = [c["offsets"].clone()]
    for k in (1, 2):
        o = list(c["off"])
        o[1], o[2] = (0, o[2]) if k == 1 else (o[3], o[3])
        offs.append(torch.tensor(o, dtype=torch.int32, device=dev()))

    def eager(o):
        c["offsets"] = o
        Y, U = forward(c)
        return (Y, U) + backward(c, U)

    ref = [eager(o) for o in offs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c["offsets"] = offs[0]
    Y, U = q.qlora_grouped_linear_fwd(c["w"], c["X"], offs[0], c["A"], c["B"], ALPHA, stream=side)
    g = q.qlora_grouped_linear_bwd(c["w"], c["X"], c["dY"], offs[0], c["A"], c["B"], ALPHA, U,
                                   stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref[0], (Y, U) + g))
    live = offs[0].clone()
    c["offsets"] = live
    out = [torch.empty_like(t) for t in ref[0]]
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            forward(c, Y=out[0], U_save=out[1])
            backward(c, out[1], dX=out[2], dA=out[3], dB=out[4])
        graphs.append(graph)
    for i in range(6):
        live.copy_(offs[i % 3])
        for t in out:
            t.fill_(3)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref[i % 3], out)), i
        c["offsets"] = offs[1]
        forward(c)
        c["offsets"] = live
        torch.cuda.synchronize()


@pytest.mark.parametrize("counts,N,K", [([2, 0, 1, 3], 272, 576), ([90, 0, 200, 31], 272, 576),
                                        ([130, 300, 257], 2080, 1088)],
                         ids=["stream", "tiles", "split_tiles"])
def test_callers_workspace(counts, N, K):
    """A workspace of exactly the size asked for, holding anything; nothing
    behind it is written, and it serves one call after another."""
    q = _api()
    c = make(counts, N, K, 32, BF)
    T, E = c["T"], len(counts)
    ref = forward(c)
    gref = backward(c, ref[1])
    for bwd in (False, True):
        n = q.qlora_grouped_linear_workspace(T, E, N, K, 32, "bf16", bwd)
        buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=dev())
        for _ in range(3):
            out = backward(c, ref[1], workspace=buf[:n]) if bwd else forward(c, workspace=buf[:n])
            assert all(torch.equal(a, b) for a, b in zip(out, gref if bwd else ref))
        assert (buf[n:] == 0xFF).all()
        with pytest.raises(q.QloraError, match="WORKSPACE"):
            backward(c, ref[1], workspace=buf[:n - 1]) if bwd else forward(c, workspace=buf[:n - 1])


def test_offsets_out_of_range_are_taken_into_the_rows():
    """Offsets past T or below 0 mean the nearest bound."""
    c = make([100, 60, 40], 272, 576, 16, BF)
    Y, U = forward(c)
    g = backward(c, U)
    c["offsets"] = torch.tensor([-5, 100, 160, 1 << 30], dtype=torch.int32, device=dev())
    Y2, U2 = forward(c)
    assert torch.equal(Y, Y2) and torch.equal(U, U2)
    assert all(torch.equal(a, b) for a, b in zip(g, backward(c, U)))


@pytest.mark.parametrize("off", [[0, 150, 20, 200], [200, 0, 300, -7], [7, 7, 3, 3]])
def test_offsets_that_decrease_stay_inside_the_buffers(off):
    """Outputs are unspecified, but nothing before or behind them is written."""
    c = make([100, 60, 40], 272, 576, 16, BF)
    c["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev())
    guarded = []

    def guard(shape, dtype):
        n = int(np.prod(shape))
        flat = torch.full((n + 8192,), 5.0, dtype=dtype, device=dev())
        guarded.append((flat, n))
        return flat[4096:4096 + n].view(shape)

    U = guard((200, 16), BF)
    forward(c, Y=guard((200, 272), BF), U_save=U)
    backward(c, U, dX=guard((200, 576), BF), dA=guard(c["A"].shape, torch.float32),
             dB=guard(c["B"].shape, torch.float32))
    for flat, n in guarded:
        assert (flat[:4096] == 5).all() and (flat[4096 + n:] == 5).all()


def test_training_step_of_routed_rows():
    """The operators as they run together: tokens sorted by expert, forward,
    backward, an AdamW step on the adapters; the step lowers what the gradient
    says it lowers (first order, exact in the 64-bit formulas)."""
    q = _api()
    c = make([40, 0, 25, 90], 144, 320, 16, BF, seed=4)
    r, lr = 16, 1e-3
    Y, U = forward(c)
    dX, dA, dB = backward(c, U)
    for name, grad in (("A", dA), ("B", dB)):
        p = c[name].float()
        before, p16 = p.clone(), torch.empty_like(c[name])
        m, v = torch.zeros_like(p), torch.zeros_like(p)
        q.qlora_adamw_step(p, m, v, grad, 1, lr, param_bf16=p16)
        # first step of Adam: lr * g / (|g| + eps'), 0 where there is no gradient
        step = host(before) - host(p)
        gd = host(grad)
        want = lr * gd / (np.abs(gd) + 1e-8)
        # three float32 roundings of a parameter below 4, and of the step
        assert (np.abs(step - want) <= 4 * 2.0 ** -23 * (np.abs(host(before)) + lr)).all()
        assert not step[1].any()                 # the expert without rows
        assert torch.equal(p16, p.to(BF))


def test_long_row_offsets():
    """T * cols close to 2^30: byte offsets past 2^31."""
    T, N, K, r = 1_000_000, 16, 1024, 16
    q = _api()
    g = torch.Generator(device=dev()).manual_seed(1)
    w = q.qlora_nf4_quantize(torch.randn(2 * N, K, generator=g, device=dev()) * 0.02)
    X = torch.zeros(T, K, dtype=BF, device=dev())
    rows = [0, 1, 499_999, 500_000, T - 200, T - 1]
    X[rows] = torch.randn(len(rows), K, generator=g, device=dev()).to(BF)
    A = (torch.randn(2, r, K, generator=g, device=dev()) / 4).to(BF)
    B = (torch.randn(2, N, r, generator=g, device=dev()) * 0.01).to(BF)
    off = [0, 500_000, T]
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    Y, U = q.qlora_grouped_linear_fwd(w, X, offsets, A, B, ALPHA)
    W = q.qlora_nf4_dequantize(w).double().view(2, N, K)
    dY = torch.zeros(T, N, dtype=BF, device=dev())
    dY[rows] = torch.randn(len(rows), N, generator=g, device=dev()).to(BF)
    dX, dA, dB = q.qlora_grouped_linear_bwd(w, X, dY, offsets, A, B, ALPHA, U)
    sel = torch.tensor(rows, device=dev())
    small = [0, sum(t < off[1] for t in rows), len(rows)]
    x, dy, u = host(X[sel]), host(dY[sel]), host(U[sel])
    a, b = host(A), host(B)
    y_ref, u_ref = grouped_forward(x, W.cpu().numpy(), a, b, small, ALPHA)
    dx_ref, da_ref, db_ref = grouped_backward(x, dy, W.cpu().numpy(), a, b, small, ALPHA, u)
    for e in range(2):
        i, j = small[e], small[e + 1]
        lim = group_bounds(x[i:j], dy[i:j], W[e].cpu().numpy(), a[e], b[e], ALPHA, HALF[BF])
        within("Y", host(Y[sel])[i:j], y_ref[i:j], lim["y"])
        within("U", u[i:j], u_ref[i:j], lim["u"])
        within("dX", host(dX[sel])[i:j], dx_ref[i:j], lim["dx"])
        within("dA", host(dA[e]), da_ref[e], lim["da"])
        within("dB", host(dB[e]), db_ref[e], db_bound(dy[i:j], u[i:j], ALPHA, r))
    Y[sel], U[sel], dX[sel] = 0, 0, 0
    assert not Y.any() and not U.any() and not dX.any()

"""Calls of the gated block and of the layer in 8-bit floating point that the
documentation allows: captured and replayed, on two streams at once, workspaces
of exactly their size, outputs of the caller's, empty batches, values that are
not finite, the longest batches; and the operators together, as a training step
and as a served block use them."""
import pytest
import torch

import fp8_ref as F
import gated_ref as R
from gpu_util import dev
from test_gpu_fp8 import tokens, weight
from test_gpu_gated import BF, HF, Case, _api, gen

pytestmark = pytest.mark.gpu


def _all(out):
    """The tensors of nested results, flat."""
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for o in out if o is not None for t in _all(o)]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(_all(a), _all(b)))


def _on(stream, f):
    with torch.cuda.stream(stream):
        return f()


class Served:
    """A gated block and the layer behind it in 8-bit floating point."""

    def __init__(self, T, N, K, dtype, seed):
        self.gate, self.up, self.down = weight(N, K, seed), weight(N, K, seed + 1), weight(K, N, seed + 2)
        self.x = tokens(T, K, dtype, seed)

    def run(self, **kw):
        q = _api()
        h = q.qlora_fp8_gated_fwd(self.gate, self.up, self.x, H=kw.get("H"),
                                  workspace=kw.get("w0"))
        return h, q.qlora_fp8_linear_fwd(self.down, h, Y=kw.get("Y"), workspace=kw.get("w1"))


SHAPES = [(3, 272, 1024, 32), (300, 528, 1088, 64), (2500, 2480, 1024, 16)]


@pytest.mark.parametrize("T,N,K,r", SHAPES)
def test_graphs(T, N, K, r):
    """Two graphs of forward and backward and of the served block, each with
    buffers and workspaces of its own, replayed in turn and on two streams, with
    eager work between."""
    q = _api()
    cs = [Case(T, N, K, r, dt, seed=s) for dt, s in (("bf16", 1), ("fp16", 2))]
    served = [Served(T, N, K, dt, s) for dt, s in ((BF, 3), (HF, 6))]
    ref = [_all((c.fwd(), c.bwd(), s.run())) for c, s in zip(cs, served)]
    torch.cuda.synchronize()
    outs, graphs, keep = [], [], []
    for c, s in zip(cs, served):
        buf = [torch.empty(n, dtype=torch.uint8, device=dev()) for n in
               (q.qlora_gated_linear_workspace(T, N, K, r, False),
                q.qlora_gated_linear_workspace(T, N, K, r, True),
                q.qlora_fp8_gated_workspace(T, N, K), q.qlora_fp8_workspace(T, K, N, False))]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = (c.fwd(workspace=buf[0]), c.bwd(workspace=buf[1]), s.run(w0=buf[2], w1=buf[3]))
        outs.append(_all(out))
        graphs.append(g)
        keep.append((buf, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(6):
        for o in outs:
            for t in o:
                t.fill_(3)
        torch.cuda.synchronize()
        for i in (0, 1):
            if k % 2:
                _on(streams[i], graphs[i].replay)
            else:
                graphs[i].replay()
        torch.cuda.synchronize()
        for o, want in zip(outs, ref):
            assert _same(o, want), k
        cs[0].bwd()
        served[1].run()
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,N,K,r", SHAPES)
def test_two_streams_at_once(T, N, K, r):
    cs = [Case(T, N, K, r, dt, seed=s) for dt, s in (("bf16", 4), ("fp16", 5))]
    served = [Served(T, N, K, dt, s) for dt, s in ((BF, 1), (HF, 9))]

    def one(i):
        return _all((cs[i].fwd(), cs[i].bwd(), served[i].run()))

    ref = [one(0), one(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            got[i].append(_on(streams[i], lambda: one(i)))
    torch.cuda.synchronize()
    assert all(_same(o, ref[i]) for i in (0, 1) for o in got[i])


def test_stream_argument():
    c = Case(130, 272, 512, 16)
    s = Served(130, 272, 512, BF, 4)
    q = _api()
    ref = _all((c.fwd(), c.bwd(), s.run()[0]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _all((c.fwd(stream=side), c.bwd(stream=side),
                q.qlora_fp8_gated_fwd(s.gate, s.up, s.x, stream=side)))
    torch.cuda.synchronize()
    assert _same(got, ref)


def _guarded(shape, dtype):
    """An output with 4096 values behind it that nobody may write."""
    n = 1
    for v in shape:
        n *= v
    flat = torch.full((n + 4096,), 5.0, dtype=dtype, device=dev())
    return flat[:n].view(shape), flat[n:]


@pytest.mark.parametrize("T,N,K,r", SHAPES + [(513, 2736, 1024, 112), (20, 528, 4288, 16)])
def test_workspace_and_outputs_of_exactly_their_size(T, N, K, r):
    """Workspaces that hold anything before, with nothing written behind them or
    behind the outputs."""
    q = _api()
    c, s = Case(T, N, K, r, "fp16"), Served(T, N, K, HF, 2)
    ref = (c.fwd(), c.bwd(), s.run())

    def buffer(n):
        return torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=dev())

    for run, sizes, shapes in (
            (lambda w, o: c.fwd(H=o[0], saved=q.GatedSaved(*o[1:]), workspace=w[0]),
             [q.qlora_gated_linear_workspace(T, N, K, r, False)],
             [(T, N)] * 3 + [(T, r)] * 2),
            (lambda w, o: c.bwd(dX=o[0], dA_gate=o[1], dB_gate=o[2], dA_up=o[3], dB_up=o[4],
                                workspace=w[0]),
             [q.qlora_gated_linear_workspace(T, N, K, r, True)],
             [(T, K), (r, K), (N, r), (r, K), (N, r)]),
            (lambda w, o: s.run(H=o[0], Y=o[1], w0=w[0], w1=w[1]),
             [q.qlora_fp8_gated_workspace(T, N, K), q.qlora_fp8_workspace(T, K, N, False)],
             [(T, N), (T, K)])):
        want = ref[2 if len(shapes) == 2 else int(shapes[0] == (T, K))]
        f32 = want is ref[1]                  # the adapters' gradients
        bufs = [buffer(n) for n in sizes]
        for _ in range(3):
            made = [_guarded(sh, torch.float32 if f32 and i else HF) for i, sh in enumerate(shapes)]
            got = run([b[:n] for b, n in zip(bufs, sizes)], [m[0] for m in made])
            assert _same(got, want)
            assert all((m[1] == 5).all() for m in made)
            assert all((b[n:] == 0xFF).all() for b, n in zip(bufs, sizes))


def test_empty_batch():
    q = _api()
    c = Case(0, 272, 512, 16)
    h, s = c.fwd()
    assert h.shape == (0, 272) and s.P_up.shape == (0, 272)
    dX, *g = c.bwd()
    assert dX.shape == (0, 512)
    assert all((t == 0).all() for t in g)
    w = weight(272, 512, 1)
    x = torch.empty(0, 512, dtype=BF, device=dev())
    assert q.qlora_fp8_gated_fwd(w, w, x).shape == (0, 272)
    assert q.qlora_fp8_linear_fwd(w, x).shape == (0, 272)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,N,K,r", [(3, 272, 1024, 32), (40, 48, 512, 16), (300, 528, 1088, 64),
                                     (513, 2736, 1024, 112), (2187, 672, 7552, 64)])
def test_values_that_are_not_finite_stay_in_their_token(T, N, K, r, bad):
    """A token's infinity or NaN reaches that token's outputs alone; in the
    backward also the sums over tokens: all of dA, and dB's row of the column it
    stands in (a reduction that ends inside a step: rows % 64 != 0)."""
    q = _api()
    c, s = Case(T, N, K, r), Served(T, N, K, BF, 5)
    t, n = T // 2, N - 1
    rest = torch.arange(T, device=dev()) != t
    rows = torch.arange(N, device=dev()) != n
    h, saved = c.fwd()
    hs = s.run()[0]
    dX, *g = c.bwd()
    keep = c.X[t, K - 1].clone(), s.x[t, K - 1].clone()
    c.X[t, K - 1] = s.x[t, K - 1] = bad
    h2, saved2 = c.fwd()
    hs2 = s.run()[0]
    assert torch.equal(h2[rest], h[rest]) and torch.equal(hs2[rest], hs[rest])
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(saved2, saved))
    assert not saved2.P_gate[t].isfinite().any() and hs2[t].isnan().all()
    c.X[t, K - 1] = keep[0]
    c.dH[t, n] = bad
    dX2, dAg, dBg, dAu, dBu = c.bwd()
    assert torch.equal(dX2[rest], dX[rest]) and not dX2[t].isfinite().any()
    assert torch.equal(dBg[rows], g[1][rows]) and torch.equal(dBu[rows], g[3][rows])
    assert not dAu.isfinite().any() and not dBu[n].isfinite().any()


def test_one_weight_and_adapter_as_both():
    """The gate and the up projection may be the same tensors."""
    c = Case(70, 272, 512, 16)
    c.w[1], c.A[1], c.B[1] = c.w[0], c.A[0], c.B[0]
    c.adapters = (c.A[0], c.B[0], c.A[0], c.B[0])
    c.check_fwd()
    c.check_bwd()


@pytest.mark.parametrize("N,K", [(16, 1024), (1024, 64)])
def test_longest_batch(N, K):
    """Byte offsets up to 2^31 in the token tensors; outputs by token, gradients
    by sums in 64 bits over chunks of the tokens."""
    q = _api()
    T, r = (2 ** 30 - 64) // 1024, 16
    print(f"[gated] longest {T} x {N} x {K}", flush=True)
    c = Case(T, N, K, r)
    w = [q.qlora_nf4_dequantize(v).double() for v in c.w]
    A, B = [v.double() for v in c.A], [v.double() for v in c.B]
    h, s = c.fwd()
    got = c.bwd()
    sums = [[0, 0], [0, 0]]
    errs = [[0, 0], [0, 0]]
    step = 2 ** 16
    for t in range(0, T, step):
        part = slice(t, min(T, t + step))
        x = c.X[part].double()
        (H, P, U), (eH, eP, eU) = R.forward(x, w, A, B, c.scale, c.act, c.dt)
        R.check(h[part], H, eH, ("H", t))
        R.check(s.P_up[part], P[1], eP[1], ("P_up", t))
        R.check(s.U_gate[part], U[0], eU[0], ("U_gate", t))
        saved = [v[part].double() for v in c.saved]
        (dX, *g), (eX, *e) = R.backward(x, c.dH[part].double(), w, A, B, c.scale, c.act, saved[:2],
                                        saved[2:], c.dt)
        R.check(got[0][part], dX, eX, ("dX", t))
        for k in range(2):
            for i in range(2):
                sums[k][i] = sums[k][i] + g[k][i]
                errs[k][i] = errs[k][i] + e[k][i]
    for k, i, y, name in ((0, 0, got[1], "dA_gate"), (1, 0, got[2], "dB_gate"),
                          (0, 1, got[3], "dA_up"), (1, 1, got[4], "dB_up")):
        # a chunk's bound counts its own sums only: T roundings instead of the
        # chunk's, of sums of magnitudes that its bound holds 2^16 times
        R.check(y, sums[k][i], errs[k][i] * (T / step), name)
        R.near(y, sums[k][i], 1e-4, name)


@pytest.mark.parametrize("T,N,K", [(2 ** 22 - 1, 3, 16), (1, 2 ** 22 - 1, 16), (20, 2 ** 20 + 3, 4112),
                                   (100, 2 ** 20 + 3, 4112), (2 ** 20 + 3, 40, 4112)])
def test_largest_8_bit_sizes(T, N, K):
    """Codes of 4 GiB and more and the longest sides: sampled outputs."""
    q = _api()
    print(f"[fp8] largest {T} x {N} x {K}", flush=True)

    def part(n, rows, k):
        return torch.randn(rows, k, generator=gen(n), device=dev()).to(BF)

    def big(n, seed):
        out = torch.empty(n, K, dtype=BF, device=dev())
        for i in range(0, n, 2 ** 18):
            out[i:i + 2 ** 18] = part(seed + i, min(n - i, 2 ** 18), K)
        return out

    W = big(N, 1)
    w = q.Fp8Weight(*q.qlora_fp8_quantize_weight(W))
    del W
    x = big(T, 2)
    y = q.qlora_fp8_linear_fwd(w, x)
    codes, scale = q.qlora_fp8_quantize(x)
    assert torch.equal(y, q.qlora_fp8_matmul(w, codes, scale)) or T <= 16
    ts = sorted({0, T // 2, T - 1} | set(range(max(0, T - 70), T)))
    ns = (N - 1) // 128 * 128
    picked = codes.view(torch.uint8)[ts].view(codes.dtype)
    for pick in (slice(0, min(N, 128)), slice(max(0, ns - 128), N)):
        blk = slice(pick.start // 128, -(-pick.stop // 128))
        ref, err = F.product(F.values(picked, scale[:, ts].T, 1),
                             F.values(w.codes[pick], w.scale[blk], 128))
        F.check(y[ts][:, pick], ref, err, (T, N, K, pick))


def test_training_step_of_a_block():
    """Gated block and the layer behind it, forward and backward as a training
    step calls them, against the same block in 64 bits, and the adapters'
    gradients against differences of the 64-bit loss.

    In norm every rounding to 16 bits of a tensor on the way (X A^T and its
    scaled copy, P twice, H, Y's seed, dH, d twice, the seeds of dX) is at most
    2^-8 of it, and a product of independent values passes a relative error of
    its factor on unchanged: ten of them."""
    q = _api()
    T, N, K, r, tol = 300, 576, 1088, 32, 10 * 2.0 ** -8
    c = Case(T, N, K, r, "bf16", act="silu")
    wd = q.qlora_nf4_quantize(torch.randn(K, N, generator=gen(8), device=dev()) * 0.05)
    Ad = (torch.randn(r, N, generator=gen(9), device=dev()) * r ** -0.5).to(BF)
    Bd = (torch.randn(K, r, generator=gen(10), device=dev()) * 0.02).to(BF)
    dY = (torch.randn(T, K, generator=gen(11), device=dev())).to(BF)
    h, saved = c.fwd()
    y, u = q.qlora_linear_fwd(wd, h, Ad, Bd, c.alpha)
    dh, dAd, dBd = q.qlora_linear_bwd(wd, h, dY, Ad, Bd, c.alpha, U_saved=u)
    dX, dAg, dBg, dAu, dBu = q.qlora_gated_linear_bwd(*c.w, c.X, dh, *c.adapters, c.alpha, saved,
                                                      act=c.act)
    x, w, A, B = c.values()
    w.append(q.qlora_nf4_dequantize(wd).double())
    leaves = [v.detach().clone().requires_grad_() for v in
              (x, A[0], B[0], A[1], B[1], Ad.double(), Bd.double())]

    def loss(x, Ag, Bg, Au, Bu, Ad, Bd):
        g = x @ w[0].T + c.scale * (x @ Ag.T) @ Bg.T
        v = x @ w[1].T + c.scale * (x @ Au.T) @ Bu.T
        h = g * torch.sigmoid(g) * v
        return ((h @ w[2].T + c.scale * (h @ Ad.T) @ Bd.T) * dY.double()).sum(), h

    out, href = loss(*leaves)
    out.backward()
    R.near(h, href.detach(), tol, "H")
    for got, leaf, name in zip((dX, dAg, dBg, dAu, dBu, dAd, dBd), leaves,
                               ("dX", "dA_gate", "dB_gate", "dA_up", "dB_up", "dA", "dB")):
        R.near(got, leaf.grad, tol, name)
    # along the gradient itself: central differences of the 64-bit loss
    with torch.no_grad():
        for i, got in ((1, dAg), (2, dBg), (3, dAu), (4, dBu)):
            v = got.double() / got.double().norm()
            e = 1e-4
            at = list(leaves)
            at[i] = leaves[i] + e * v
            hi = loss(*at)[0]
            at[i] = leaves[i] - e * v
            slope = (hi - loss(*at)[0]) / (2 * e)
            assert abs(slope - (got.double() * v).sum()) <= 2 * tol * abs(slope), (i, slope)


@pytest.mark.parametrize("T", [1, 24, 300])
def test_serving_a_merged_block(T):
    """Adapters merged, weights quantised to 8 bits, the block and the layer
    behind it on 16-bit tokens: each half against its formula, and the whole
    against the unmerged block.

    Codes are off by at most 2^-4 relative, so in norm a projection by sqrt(2)
    2^-4 (its two factors, independently), H by at most 1.1 sqrt(2) of that (two
    projections; the activation's slope is at most 1.1), and Y by H's error and its
    own: sqrt((1.1 * 2 * 2^-4)^2 + 2 * 2^-8) = 0.164."""
    q = _api()
    N, K, r = 576, 1088, 32
    c = Case(T, N, K, r, "bf16", act="silu")
    wd = q.qlora_nf4_quantize(torch.randn(K, N, generator=gen(8), device=dev()) * 0.05)
    Ad = (torch.randn(r, N, generator=gen(9), device=dev()) * r ** -0.5).to(BF)
    Bd = (torch.randn(K, r, generator=gen(10), device=dev()) * 0.02).to(BF)
    gate, up = (q.Fp8Weight(*q.qlora_fp8_quantize_weight(q.qlora_nf4_merge(w, a, b, c.alpha)))
                for w, a, b in zip(c.w, c.A, c.B))
    down = q.Fp8Weight(*q.qlora_fp8_quantize_weight(q.qlora_nf4_merge(wd, Ad, Bd, c.alpha)))
    h = q.qlora_fp8_gated_fwd(gate, up, c.X, act=c.act)
    y = q.qlora_fp8_linear_fwd(down, h)
    codes, scale = q.qlora_fp8_quantize(c.X)
    ref, err = F.gated(F.values(codes, scale.T, 1), F.values(gate.codes, gate.scale, 128),
                       F.values(up.codes, up.scale, 128), c.act)
    F.check(h, ref, err, ("H", T))
    codes, scale = q.qlora_fp8_quantize(h)
    F.check(y, *F.product(F.values(codes, scale.T, 1), F.values(down.codes, down.scale, 128)),
            ("Y", T))
    hu, _ = c.fwd(save=False)
    yu, _ = q.qlora_linear_fwd(wd, hu, Ad, Bd, c.alpha)
    R.near(y, yu.double(), 0.164 + 2.0 ** -6, "Y")

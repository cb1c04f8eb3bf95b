"""The linear layer in 8-bit integers on the GPU: codes and scales equal to
the exact rule bit for bit, products within their few roundings of the exact
integer sums."""
import numpy as np
import pytest
import torch

from gpu_util import dev, f32_dev

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11}       # half a step relative to the value


def _api():
    import bit_nf4_quantized_06_amd as q
    return q


def codes_ref(x):
    """float64 rule: x holds values of at most 24 bits, so quotient and rint in
    float64 decide every border between two codes exactly (a quotient that is
    not half-way differs from it by more than 2^-32)."""
    x = x.astype(np.float64)
    scale = (np.abs(x).max(1) / 127).astype(np.float32)
    s = scale.astype(np.float64)[:, None]
    code = np.where(s > 0, np.rint(x / np.where(s > 0, s, 1)), 0)
    return np.clip(code, -127, 127).astype(np.int8), scale


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


@pytest.mark.parametrize("dtype", [BF, HF, FF], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (130, 512), (5, 2064), (3, 4096),
                                       (2, 9216), (7, 22016), (3, 40000), (2, 131056)])
def test_quantize_is_exact(rows, cols, dtype):
    print(f"[int8] quantize {rows} x {cols} {dtype}", flush=True)
    x = torch.randn(rows, cols, generator=gen(rows * cols), device=dev()) * 3
    if rows > 2:
        x[1] = 0                         # a row of zeros
        x[2] = x[2].sign() * 2.5         # equal magnitudes
    x[0, : 8] = torch.tensor([127, 0.5, -0.5, 1.5, 2.5, -126.5, 126.5, 3.5], device=dev())
    x[0, 8:] = x[0, 8:].clamp(-127, 127)  # scale 1: the halves are exact ties
    x = x.to(dtype)
    codes, scale = _api().qlora_int8_quantize(x)
    ref_c, ref_s = codes_ref(x.float().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), ref_s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), ref_c)
    assert ref_s[0] == 1.0 and list(ref_c[0, :8]) == [127, 0, 0, 2, 2, -126, 126, 4]


def test_quantize_tiny_and_large_rows():
    """Rows whose scale is subnormal, underflows to 0, or is near the largest
    float32."""
    x = torch.randn(6, 64, generator=gen(1), device=dev())
    x = x * torch.tensor([1e-37, 1e-39, 1e-43, 1e-45, 1e37, 1.0], device=dev())[:, None]
    codes, scale = _api().qlora_int8_quantize(x)
    ref_c, ref_s = codes_ref(x.cpu().numpy())
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), ref_s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), ref_c)


@pytest.mark.parametrize("dtype", [BF, HF, FF], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [16, 1024, 9216, 131056])
def test_rows_that_are_not_finite(cols, dtype):
    """An infinity or a NaN anywhere in a row: codes 0 and that scale, in that
    row alone; its outputs are NaN, at every number of tokens."""
    q = _api()
    x = torch.randn(7, cols, generator=gen(cols), device=dev())
    x[1, cols // 2] = float("inf")
    x[2, cols - 1] = float("nan")
    x[4, 0] = float("nan")
    x[4, cols - 3] = float("-inf")
    x = x.to(dtype)
    if dtype == FF:                     # a NaN whose low bits are set
        x.view(torch.int32)[2, cols - 1] = -5
    codes, scale = q.qlora_int8_quantize(x)
    good = [0, 3, 5, 6]
    ref_c, ref_s = codes_ref(x[good].float().cpu().numpy())
    assert np.array_equal(codes[good].cpu().numpy(), ref_c)
    assert np.array_equal(scale[good].cpu().numpy(), ref_s)
    assert not codes[[1, 2, 4]].any()
    assert scale[1].isinf() and scale[[2, 4]].isnan().all()
    if dtype == FF or cols > 9216:
        return
    W, ws, _, _ = product_case(1, 33, cols, 5)
    w = q.Int8Weight(W, ws)
    for rows in (slice(0, 3), slice(0, 7)):
        y = q.qlora_int8_linear_fwd(w, x[rows].contiguous())
        bad = [i for i in (1, 2, 4) if i < len(y)]
        rest = [i for i in good if i < len(y)]
        assert y[bad].isnan().all()
        check_product(y[rest], W, ws, codes[rest], scale[rest], (cols, dtype))


def product_case(T, N, K, seed):
    g = gen(seed)
    W = torch.randint(-127, 128, (N, K), generator=g, device=dev(), dtype=torch.int8)
    X = torch.randint(-127, 128, (T, K), generator=g, device=dev(), dtype=torch.int8)
    ws = torch.rand(N, generator=g, device=dev()) * 1e-3 + 1e-4
    xs = torch.rand(T, generator=g, device=dev()) * 1e-2 + 1e-3
    return W, ws, X, xs


def check_product(y, W, ws, X, xs, what):
    """The integer sum is exact; it is converted to float32 (2^-24 relative),
    multiplied twice (2^-24 each) and rounded to 16 bits: half a step, which
    for fp16 below its normal range is 2^-25 at least."""
    acc = X.double() @ W.double().T             # below 2^53: exact
    ref = acc * ws.double() * xs.double()[:, None]
    lim = (HALF[y.dtype] + 3.01 * 2.0 ** -24) * ref.abs() + (2.0 ** -25 if y.dtype == HF else 0)
    bad = (y.double() - ref).abs() > lim
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


SIZES = [(1, 1, 16), (1, 4096, 4096), (2, 100, 144), (16, 1000, 4096), (17, 33, 2064),
         (33, 257, 11008), (64, 512, 1040), (5, 48, 131056), (65, 128, 128), (65, 1, 16),
         (128, 128, 256), (129, 130, 272), (200, 1001, 1040), (300, 333, 4112),
         (211, 4096, 11008), (1000, 1100, 2048), (700, 777, 6160), (2000, 9000, 640),
         (4500, 4612, 1168), (70, 40, 131056),
         # the four tiles whole and split, each with a ragged last step
         (600, 5000, 11024), (211, 4096, 11024), (1300, 3001, 1040), (400, 3001, 11024),
         (1300, 3001, 8208), (640, 8192, 22032), (1300, 6003, 1040), (1500, 3001, 22032),
         (1500, 1500, 16400), (700, 1500, 11024)]


@pytest.mark.parametrize("T,N,K", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_product(T, N, K):
    q = _api()
    print(f"[int8] product {T} x {N} x {K}", flush=True)
    W, ws, X, xs = product_case(T, N, K, T + N)
    w = q.Int8Weight(W, ws)
    for dtype in (BF, HF):
        Y = torch.full((T + 1, N), 7.0, dtype=dtype, device=dev())
        y = q.qlora_int8_matmul(w, X, xs, dtype=dtype, Y=Y[:T])
        check_product(y, W, ws, X, xs, (T, N, K, dtype))
        assert (Y[T] == 7).all()                # the row behind the last
        again = q.qlora_int8_matmul(w, X, xs, dtype=dtype)
        assert torch.equal(again, y)


@pytest.mark.parametrize("T,N,K", [(3, 64, 64), (70, 96, 1040), (400, 2100, 512), (3, 16, 131056),
                                   (90, 130, 131056)])
def test_extreme_codes(T, N, K):
    """Every product 127 * 127 (and -128 * -128): the largest sums."""
    q = _api()
    for v in (127, -128):
        W = torch.full((N, K), v, dtype=torch.int8, device=dev())
        X = torch.full((T, K), v, dtype=torch.int8, device=dev())
        ws, xs = torch.full((N,), 1e-3, device=dev()), torch.full((T,), 1e-3, device=dev())
        y = q.qlora_int8_matmul(q.Int8Weight(W, ws), X, xs)
        check_product(y, W, ws, X, xs, v)


@pytest.mark.parametrize("T", [1, 2, 5, 16, 40, 64, 65, 150, 700])
@pytest.mark.parametrize("N,K", [(272, 1040), (1024, 4096), (48, 22016)])
def test_linear_is_quantize_then_product(T, N, K):
    q = _api()
    print(f"[int8] linear {T} x {N} x {K}", flush=True)
    for dtype in (BF, HF):
        x = torch.randn(T, K, generator=gen(T), device=dev()).to(dtype)
        if T > 1:
            x[1] = 0
        W, ws, _, _ = product_case(1, N, K, 5)
        w = q.Int8Weight(W, ws)
        y = q.qlora_int8_linear_fwd(w, x)
        codes, xs = q.qlora_int8_quantize(x)
        assert torch.equal(y, q.qlora_int8_matmul(w, codes, xs, dtype=dtype))
        check_product(y, W, ws, codes, xs, (T, N, K, dtype))


def test_zero_scales_and_empty_batches():
    q = _api()
    W, ws, X, xs = product_case(20, 64, 64, 2)
    ws[3] = 0
    xs[4] = 0
    y = q.qlora_int8_matmul(q.Int8Weight(W, ws), X, xs)
    assert (y[:, 3] == 0).all() and (y[4] == 0).all()
    w = q.Int8Weight(W, ws)
    assert q.qlora_int8_linear_fwd(w, torch.empty(0, 64, dtype=BF, device=dev())).shape == (0, 64)
    assert q.qlora_int8_matmul(w, X[:0], xs[:0]).shape == (0, 64)
    c, s = q.qlora_int8_quantize(torch.empty(0, 64, device=dev()))
    assert c.shape == (0, 64) and s.shape == (0,)


def test_served_from_a_merged_weight():
    """The deployment run: NF4 weight, adapter merged, merged weight in 8
    bits, tokens through it.  Against 64 bits: every weight and token is off
    by at most half a code step, so an output is off by at most
    sum (|x| dw + |w| dx + dx dw) with dw = w_scale / 2, dx = x_scale / 2
    (codes of exact quotients: half a step), then the product's roundings."""
    q = _api()
    N, K, r, T = 272, 1024, 16, 37
    g = gen(9)
    W = torch.randn(N, K, generator=g, device=dev()) * 0.02
    A = (torch.randn(r, K, generator=g, device=dev()) * 0.25).to(BF)
    B = (torch.randn(N, r, generator=g, device=dev()) * 0.01).to(BF)
    merged = q.qlora_nf4_merge(q.qlora_nf4_quantize(W), A, B, 16.0)
    w = q.Int8Weight(*q.qlora_int8_quantize(merged))
    x = torch.randn(T, K, generator=g, device=dev()).to(BF)
    y = q.qlora_int8_linear_fwd(w, x).double()
    _, xs = q.qlora_int8_quantize(x)
    wd, xd = merged.double(), x.double()
    ref = xd @ wd.T
    dw, dx = w.scale.double()[None, :] / 2, xs.double()[:, None] / 2
    lim = (xd.abs().sum(1)[:, None] * dw + wd.abs().sum(1)[None] * dx + K * dw * dx) * 1.0001
    assert ((y - ref).abs() <= lim + 1.01 * HALF[BF] * (ref.abs() + lim)).all()


@pytest.mark.parametrize("T", [1, 30, 300])
def test_streams_and_graph(T):
    """On a stream of the caller's while another is current, and captured:
    each replay on new inputs equals the eager call."""
    q = _api()
    N, K = 1040, 2064
    W, ws, _, _ = product_case(1, N, K, 3)
    w = q.Int8Weight(W, ws)
    xs = [torch.randn(T, K, generator=gen(i), device=dev()).to(BF) for i in range(4)]
    ref = [q.qlora_int8_linear_fwd(w, x) for x in xs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [q.qlora_int8_linear_fwd(w, x, stream=side[i % 2]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    x = xs[0].clone()
    Y = torch.empty(T, N, dtype=BF, device=dev())
    graphs = []
    for _ in range(2):                    # two graphs of the same call
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.qlora_int8_linear_fwd(w, x, Y=Y)
        graphs.append(g)
    for i in range(6):
        x.copy_(xs[i % 4])
        Y.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref[i % 4]), i
        q.qlora_int8_linear_fwd(w, xs[1])   # the program's own work between replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,N,K", [(2 ** 22 - 1, 3, 16), (1, 2 ** 22 - 1, 16),
                                   (70, 2 ** 22 - 1, 16), (2 ** 20, 100, 64)])
def test_largest_rows(T, N, K):
    q = _api()
    print(f"[int8] largest {T} x {N} x {K}", flush=True)
    W, ws, X, xs = product_case(T, N, K, 11)
    w = q.Int8Weight(W, ws)
    y = q.qlora_int8_matmul(w, X, xs)
    for t in range(0, T, 2 ** 20):
        for n in range(0, N, 2 ** 20):
            check_product(y[t:t + 2 ** 20, n:n + 2 ** 20], W[n:n + 2 ** 20], ws[n:n + 2 ** 20],
                          X[t:t + 2 ** 20], xs[t:t + 2 ** 20], (T, N, K, t, n))
    x = X.to(BF)
    codes, scale = q.qlora_int8_quantize(x)
    assert torch.equal(q.qlora_int8_linear_fwd(w, x), q.qlora_int8_matmul(w, codes, scale))
    rows = [0, T // 2, T - 1]
    ref_c, ref_s = codes_ref(x[rows].float().cpu().numpy())
    assert np.array_equal(codes[rows].cpu().numpy(), ref_c)
    assert np.array_equal(scale[rows].cpu().numpy(), ref_s)


@pytest.mark.parametrize("T,N,K", [(1, 272, 1040), (20, 1040, 2064), (300, 333, 4112),
                                   (640, 8192, 4112)])
def test_callers_workspace(T, N, K):
    """A workspace of exactly the size asked for, holding anything; nothing
    behind it is written, and it serves one call after another."""
    q = _api()
    W, ws, X, xs = product_case(T, N, K, 7)
    w = q.Int8Weight(W, ws)
    x = torch.randn(T, K, generator=gen(T), device=dev()).to(BF)
    for given, call in ((True, lambda **kw: q.qlora_int8_matmul(w, X, xs, **kw)),
                        (False, lambda **kw: q.qlora_int8_linear_fwd(w, x, **kw))):
        n = q.qlora_int8_workspace(T, N, K, given)
        buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=dev())
        ref = call()
        for _ in range(3):
            assert torch.equal(call(workspace=buf[:n]), ref)
        assert (buf[n:] == 0xFF).all()
        if n:
            with pytest.raises(q.QloraError, match="WORKSPACE"):
                call(workspace=buf[:n - 1])


def test_unaligned_rows_are_refused():
    q = _api()
    W, ws, X, xs = product_case(20, 64, 64, 2)
    flat = torch.zeros(20 * 64 + 8, dtype=BF, device=dev())
    x = flat[4:4 + 20 * 64].view(20, 64)            # 8 bytes past a 16-byte border
    with pytest.raises(q.QloraError, match="ALIGN"):
        q.qlora_int8_linear_fwd(q.Int8Weight(W, ws), x)
    with pytest.raises(q.QloraError, match="ALIGN"):
        q.qlora_int8_quantize(x)
    with pytest.raises(ValueError):
        q.qlora_int8_matmul(q.Int8Weight(W, ws), X.cpu(), xs)
    assert f32_dev(np.zeros(1)).is_cuda

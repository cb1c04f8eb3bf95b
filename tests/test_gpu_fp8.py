"""The linear layer and the gated block in 8-bit floating point on the GPU:
codes and scales equal to the rule bit for bit, products within the rounding
errors of their float32 sums."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn
IDS = {BF: "bf16", HF: "fp16", FF: "fp32"}


def _api():
    import bit_nf4_quantized_06_amd as q
    return q


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def same_codes(x, codes, scale, br):
    """scale as the row blocks by column blocks"""
    c, s = R.quantize(x.float().cpu().numpy(), br)
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(codes.float().cpu().numpy(), c.astype(np.float32))


@pytest.mark.parametrize("dtype", [BF, HF, FF], ids=IDS.get)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (130, 512), (5, 2064), (257, 1040),
                                       (2, 9216), (7, 22016), (2, 131056)])
def test_quantize_is_exact(rows, cols, dtype):
    q = _api()
    print(f"[fp8] quantize {rows} x {cols} {dtype}", flush=True)
    x = torch.randn(rows, cols, generator=gen(rows * cols), device=dev()) * 3
    if rows > 2:
        x[1] = 0                          # a row of zeros
        x[2] = x[2].sign() * 2.5          # equal magnitudes
    # scale 1 in the first block: borders between codes, one of them subnormal,
    # and their neighbours
    x[0, :16] = torch.tensor([448, 17, 18, 19, -17, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10,
                              -5 * 2.0 ** -10, 432, 416, 424, 2.0 ** -9, 0.5, -448], device=dev())
    x[0, 16:128] = x[0, 16:128].clamp(-448, 448)
    x = x.to(dtype)
    codes, scale = q.qlora_fp8_quantize(x)
    assert codes.dtype == E4 and scale.shape == (-(-cols // 128), rows)
    same_codes(x, codes, scale.T, 1)
    assert scale[0, 0] == 1.0
    assert codes[0, :16].float().tolist() == [448, 16, 18, 20, -16, 1.0, 1.25, 0, 2.0 ** -8,
                                              -2.0 ** -8, 448, 416, 416, 2.0 ** -9, 0.5, -448]
    codes, scale = q.qlora_fp8_quantize_weight(x)
    assert scale.shape == (-(-rows // 128), -(-cols // 128))
    same_codes(x, codes, scale, 128)


def test_quantize_borders():
    """Quotients next to every border of E4M3: x is the border times an odd
    scale, and its neighbours in float32."""
    q = _api()
    mids = (R.E4M3[1:] + R.E4M3[:-1]) / 2
    rows = []
    for s in (1.0, 1.2345678, 0.7654321, 1.9999999, 3.1e-5, 7.7e20, 1.0000001):
        s = float(np.float32(s))
        top = np.float32(448 * s)
        s = float(np.float32(np.float64(top) / 448))
        m = (mids * s).astype(np.float32)
        for v in (m, np.nextafter(m, np.float32(np.inf)), np.nextafter(m, np.float32(0))):
            row = np.zeros(128, np.float32)
            row[:126], row[127] = v, top
            rows += [row, -row]
    x = torch.from_numpy(np.array(rows)).to(dev())
    codes, scale = q.qlora_fp8_quantize(x)
    same_codes(x, codes, scale.T, 1)


def test_quantize_tiny_and_large_blocks():
    """Blocks whose scale is subnormal, underflows to 0, or is near the largest
    float32."""
    q = _api()
    x = torch.randn(9, 256, generator=gen(1), device=dev())
    x = x * torch.tensor([1e-21, 1e-24, 1e-34, 1e-37, 1e-40, 1e-43, 1e-45, 1e37, 1.0],
                         device=dev())[:, None]
    codes, scale = q.qlora_fp8_quantize(x)
    same_codes(x, codes, scale.T, 1)
    for i in range(len(x)):
        w = x[i].view(2, 128).contiguous()
        codes, scale = q.qlora_fp8_quantize_weight(w)
        same_codes(w, codes, scale, 128)


@pytest.mark.parametrize("dtype", [BF, HF, FF], ids=IDS.get)
def test_blocks_that_are_not_finite(dtype):
    """An infinity or a NaN: codes 0 and that scale, in its block alone; its
    token's outputs are NaN and nobody else's, at every number of tokens."""
    q = _api()
    K = 400
    for T in (5, 70):
        x = torch.randn(T, K, generator=gen(T), device=dev())
        x[1, 200] = float("inf")
        x[2, 399] = float("nan")
        x = x.to(dtype)
        codes, scale = q.qlora_fp8_quantize(x)
        hit = torch.zeros(T, K, dtype=torch.bool, device=dev())
        hit[1, 128:256] = True
        hit[2, 384:] = True
        assert not codes.float()[hit].any()
        assert scale[1, 1].isinf() and scale[3, 2].isnan()
        clean = x.float().masked_fill(hit, 0)
        c, s = R.quantize(clean.cpu().numpy(), 1)
        assert np.array_equal(codes.float().cpu().numpy(), c.astype(np.float32))
        keep = ~hit[:, ::128].T.contiguous()
        assert np.array_equal(scale[keep].cpu().numpy(), s.T[keep.cpu().numpy()])
        if dtype == FF:
            continue
        w = q.Fp8Weight(*q.qlora_fp8_quantize_weight(
            torch.randn(33, K, generator=gen(3), device=dev())))
        for y in (q.qlora_fp8_linear_fwd(w, x), q.qlora_fp8_gated_fwd(w, w, x)):
            assert y[1:3].isnan().all()
            rest = [0] + list(range(3, T))
            assert y[rest].isfinite().all()


def weight(rows, cols, seed):
    q = _api()
    w = torch.randn(rows, cols, generator=gen(seed), device=dev()) * 0.02
    return q.Fp8Weight(*q.qlora_fp8_quantize_weight(w))


def tokens(T, cols, dtype, seed):
    x = torch.randn(T, cols, generator=gen(seed), device=dev())
    wide = torch.rand(cols, generator=gen(seed + 1), device=dev()) < 0.01
    return torch.where(wide, 8 * x, x).to(dtype)


SIZES = [(1, 1, 16), (1, 4096, 4096), (2, 100, 144), (16, 1000, 4096), (17, 33, 2064),
         (33, 257, 11008), (64, 512, 1040), (5, 48, 131056), (65, 128, 128), (65, 1, 16),
         (100, 130, 272), (211, 1024, 11008), (129, 4100, 400), (300, 770, 1296), (513, 2048, 640),
         (1000, 1001, 4096), (2100, 2752, 1024), (8192, 640, 384)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=IDS.get)
@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear(T, N, K, dtype):
    q = _api()
    print(f"[fp8] linear {T} x {N} x {K} {dtype}", flush=True)
    w = weight(N, K, N + K)
    x = tokens(T, K, dtype, T)
    codes, scale = q.qlora_fp8_quantize(x)
    ref, err = R.product(R.values(codes, scale.T, 1), R.values(w.codes, w.scale, 128))
    y = q.qlora_fp8_matmul(w, codes, scale, dtype=dtype)
    R.check(y, ref, err, (T, N, K))
    assert torch.equal(y, q.qlora_fp8_matmul(w, codes, scale, dtype=dtype))
    R.check(q.qlora_fp8_linear_fwd(w, x), ref, err, (T, N, K))


@pytest.mark.parametrize("dtype", [BF, HF], ids=IDS.get)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gated(T, N, K, act, dtype):
    q = _api()
    print(f"[fp8] gated {T} x {N} x {K} {dtype}", flush=True)
    gate, up = weight(N, K, N + K), weight(N, K, N + K + 1)
    x = tokens(T, K, dtype, T)
    codes, scale = q.qlora_fp8_quantize(x)
    ref, err = R.gated(R.values(codes, scale.T, 1), R.values(gate.codes, gate.scale, 128),
                       R.values(up.codes, up.scale, 128), act)
    h = q.qlora_fp8_gated_fwd(gate, up, x, act=act)
    R.check(h, ref, err, (T, N, K, act))
    assert torch.equal(h, q.qlora_fp8_gated_fwd(gate, up, x, act=act))

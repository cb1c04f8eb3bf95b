"""The row quantiser next to the borders between codes, where its fast path
hands over to the exact rule: bit for bit the 64-bit rule, in every kernel."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_int8 import _api, codes_ref, product_case

pytestmark = pytest.mark.gpu

DELTAS = np.array([0, 1e-7, 1e-6, 1e-5, 1.9e-5, 3.9e-5, 3.99e-5, 4e-5, 4.01e-5, 4.1e-5, 1e-4])


def border_matrix(rows, cols, dtype, seed, alone):
    """Rows of any scale whose elements lie (k + 1/2 + delta) scales from 0.
    alone: at most one such element in every 16, so the others of its vector
    would all take the fast path."""
    rng = np.random.default_rng(seed)
    top = (1 + rng.random(rows)) * np.exp2(rng.integers(-90, 90, rows) if dtype == torch.float32
                                           else rng.integers(-8, 8, rows))
    top = torch.from_numpy(top.astype(np.float32)).to(dtype).float().numpy()
    s = (np.abs(top.astype(np.float64)) / 127).astype(np.float32).astype(np.float64)[:, None]
    k = rng.integers(-126, 126, (rows, cols))
    off = rng.choice(DELTAS, (rows, cols)) * rng.choice([-1, 1], (rows, cols)) + 0.5
    if alone:
        off = np.where(np.arange(cols) % 16 == rng.integers(0, 16, (rows, 1)), off, 0.125)
    x = ((k + off) * s).astype(np.float32)
    x[:, 3] = top
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("alone", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16],
                         ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(700, 1024), (3, 48), (9, 9216), (2, 131056), (700, 4096)])
def test_codes_at_borders(rows, cols, dtype, alone):
    print(f"[int8] borders {rows} x {cols} {dtype} {alone}", flush=True)
    x = border_matrix(rows, cols, dtype, rows + cols, alone)
    codes, scale = _api().qlora_int8_quantize(x.to(dev()))
    ref_c, ref_s = codes_ref(x.float().numpy())
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), ref_s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), ref_c)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_codes_at_borders_inside_the_streaming_kernel(dtype):
    """Tokens quantised within the product give the product of the quantiser's
    codes; weights of one 1 a row read the codes back."""
    q = _api()
    for T, K in ((1, 4096), (2, 1040), (5, 272)):
        x = border_matrix(T, K, dtype, T + K, False).to(dev())
        W, ws, _, _ = product_case(1, 48, K, 5)
        W[:16] = 0
        W[torch.arange(16), torch.randperm(K, generator=torch.Generator().manual_seed(K))[:16]] = 1
        w = q.Int8Weight(W, ws)
        codes, xs = q.qlora_int8_quantize(x)
        assert torch.equal(q.qlora_int8_linear_fwd(w, x),
                           q.qlora_int8_matmul(w, codes, xs, dtype=dtype))

"""Every tile of the 8-bit product, whole and split, with ragged tokens,
outputs and reduction; the form each size takes is asserted without a GPU in
test_plans_cpu.py."""
import pytest
import torch

from test_gpu_int8 import BF, HF, _api, check_product, product_case

pytestmark = pytest.mark.gpu

FORM_SIZES = [(1100, 2003, 7072), (333, 8195, 6288), (211, 4098, 8768), (333, 3001, 9392),
              (70, 6003, 10592), (1400, 3001, 2128), (1400, 4098, 8352), (1500, 6003, 2368),
              (900, 8195, 1856), (300, 1001, 8272), (70, 500, 10800), (700, 2003, 352),
              (1500, 1501, 16400), (1500, 3002, 22032), (640, 8195, 22032), (500, 8194, 22032),
              (15, 1003, 4112), (31, 2050, 2064), (63, 515, 1040)]


@pytest.mark.parametrize("T,N,K", FORM_SIZES, ids=["x".join(map(str, s)) for s in FORM_SIZES])
def test_product_form(T, N, K):
    q = _api()
    print(f"[int8] product {T} x {N} x {K}", flush=True)
    W, ws, X, xs = product_case(T, N, K, T + N)
    w = q.Int8Weight(W, ws)
    for dtype in (BF, HF):
        Y = torch.full((T + 1, N), 7.0, dtype=dtype, device=W.device)
        y = q.qlora_int8_matmul(w, X, xs, dtype=dtype, Y=Y[:T])
        check_product(y, W, ws, X, xs, (T, N, K, dtype))
        assert (Y[T] == 7).all()

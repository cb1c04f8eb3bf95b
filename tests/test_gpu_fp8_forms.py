"""Every tile of the product in 8-bit floating point, whole and split, of one
weight and of a gated block, with ragged tokens, outputs and reduction; the form
each size takes is asserted without a GPU in test_gated_plans_cpu.py."""
import pytest
import torch

import fp8_ref as R
from test_gpu_fp8 import BF, HF, IDS, _api, tokens, weight

pytestmark = pytest.mark.gpu

FORM_SIZES = [(1247, 5267, 16), (2, 6929, 15760), (408, 2601, 15008), (2775, 1577, 976),
              (1100, 2003, 7072), (70, 6003, 10592), (1500, 6003, 2368), (1154, 3365, 18592),
              (1, 7633, 20976), (65, 515, 16 * 1025)]
GATED_FORM_SIZES = [(1375, 2213, 16), (390, 1297, 13104), (138, 3138, 20672), (578, 3329, 1008),
                    (1, 4203, 14000), (900, 515, 16016), (2017, 3291, 144), (516, 3569, 15920),
                    (1, 3761, 15920), (65, 515, 16 * 1025)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=IDS.get)
@pytest.mark.parametrize("T,N,K", FORM_SIZES, ids=["x".join(map(str, s)) for s in FORM_SIZES])
def test_product_form(T, N, K, dtype):
    q = _api()
    print(f"[fp8] product {T} x {N} x {K} {dtype}", flush=True)
    w = weight(N, K, T + N)
    x = tokens(T, K, dtype, T)
    codes, scale = q.qlora_fp8_quantize(x)
    ref, err = R.product(R.values(codes, scale.T, 1), R.values(w.codes, w.scale, 128))
    Y = torch.full((T + 1, N), 7.0, dtype=dtype, device=x.device)
    y = q.qlora_fp8_matmul(w, codes, scale, dtype=dtype, Y=Y[:T])
    R.check(y, ref, err, (T, N, K))
    assert (Y[T] == 7).all()
    Y.fill_(7.0)
    R.check(q.qlora_fp8_linear_fwd(w, x, Y=Y[:T]), ref, err, (T, N, K))
    assert (Y[T] == 7).all()


@pytest.mark.parametrize("dtype,act", [(BF, "gelu_tanh"), (HF, "silu")], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", GATED_FORM_SIZES,
                         ids=["x".join(map(str, s)) for s in GATED_FORM_SIZES])
def test_gated_form(T, N, K, dtype, act):
    q = _api()
    print(f"[fp8] gated {T} x {N} x {K} {dtype}", flush=True)
    gate, up = weight(N, K, T + N), weight(N, K, T + N + 1)
    x = tokens(T, K, dtype, T)
    codes, scale = q.qlora_fp8_quantize(x)
    ref, err = R.gated(R.values(codes, scale.T, 1), R.values(gate.codes, gate.scale, 128),
                       R.values(up.codes, up.scale, 128), act)
    H = torch.full((T + 1, N), 7.0, dtype=dtype, device=x.device)
    R.check(q.qlora_fp8_gated_fwd(gate, up, x, act=act, H=H[:T]), ref, err, (T, N, K, act))
    assert (H[T] == 7).all()

"""The gated feed-forward block over NF4 weights on the GPU against the formulas
in 64 bits: both directions, ragged sizes, ranks, formats, the streaming, the
tiled and the once-dequantised paths and split tiles."""
import pytest
import torch

import gated_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
DT = {"bf16": BF, "fp16": HF}


def _api():
    import bit_nf4_quantized_06_amd as q
    return q


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


class Case:
    def __init__(self, T, N, K, r, dtype="bf16", dq=True, act="silu", alpha=16.0, seed=0):
        q = _api()
        self.dims, self.dt, self.act, self.alpha = (T, N, K, r), DT[dtype], act, alpha
        self.scale, g = alpha / r, gen(seed + T + N + K + r)

        def rand(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=dev()) * std).to(self.dt)

        self.w = [q.qlora_nf4_quantize(torch.randn(N, K, generator=g, device=dev()) * 0.05,
                                       double_quant=dq, compute_dtype=dtype) for _ in range(2)]
        self.X = rand(T, K)
        self.A = [rand(r, K, std=r ** -0.5) for _ in range(2)]
        self.B = [rand(N, r, std=0.02) for _ in range(2)]
        self.dH = rand(T, N, std=2.0 ** -5)
        self.saved = q.GatedSaved(rand(T, N, std=1.5), rand(T, N, std=1.5), rand(T, r, std=2.0),
                                  rand(T, r, std=2.0))
        self.adapters = (self.A[0], self.B[0], self.A[1], self.B[1])

    def values(self):
        q = _api()
        return (self.X.double(), [q.qlora_nf4_dequantize(w).double() for w in self.w],
                [a.double() for a in self.A], [b.double() for b in self.B])

    def fwd(self, **kw):
        return _api().qlora_gated_linear_fwd(*self.w, self.X, *self.adapters, self.alpha,
                                             act=self.act, **kw)

    def bwd(self, **kw):
        return _api().qlora_gated_linear_bwd(*self.w, self.X, self.dH, *self.adapters, self.alpha,
                                             self.saved, act=self.act, **kw)

    def check_fwd(self):
        x, w, A, B = self.values()
        (H, P, U), (eH, eP, eU) = R.forward(x, w, A, B, self.scale, self.act, self.dt)
        h, s = self.fwd()
        for got, ref, err, name in ((h, H, eH, "H"), (s.P_gate, P[0], eP[0], "P_gate"),
                                    (s.P_up, P[1], eP[1], "P_up"), (s.U_gate, U[0], eU[0], "U_gate"),
                                    (s.U_up, U[1], eU[1], "U_up")):
            R.check(got, ref, err, (name, self.dims))
            R.near(got, ref, 5e-3, (name, self.dims))
        only, none = self.fwd(save=False)
        assert none is None and torch.equal(only, h)

    def check_bwd(self):
        x, w, A, B = self.values()
        s = [t.double() for t in self.saved]
        (dX, dA, dB), (eX, eA, eB) = R.backward(x, self.dH.double(), w, A, B, self.scale, self.act,
                                                s[:2], s[2:], self.dt)
        got = self.bwd()
        for y, ref, err, name, tol in ((got[0], dX, eX, "dX", 5e-3),
                                       (got[1], dA[0], eA[0], "dA_gate", 1e-5),
                                       (got[2], dB[0], eB[0], "dB_gate", 1e-5),
                                       (got[3], dA[1], eA[1], "dA_up", 1e-5),
                                       (got[4], dB[1], eB[1], "dB_up", 1e-5)):
            R.check(y, ref, err, (name, self.dims))
            R.near(y, ref, tol, (name, self.dims))
        again = self.bwd()
        assert all(torch.equal(a, b) for a, b in zip(got, again))


SMALL = [(1, 16, 64, 16), (2, 272, 128, 32), (16, 1008, 512, 48), (17, 64, 2048, 16),
         (33, 176, 320, 64), (64, 512, 1024, 128), (65, 16, 64, 16), (100, 144, 256, 16),
         (257, 400, 192, 80), (600, 1040, 448, 64), (513, 2736, 1024, 112)]


@pytest.mark.parametrize("dtype,dq,act", [("bf16", True, "silu"), ("bf16", False, "gelu_tanh"),
                                          ("fp16", True, "gelu_tanh"), ("fp16", False, "silu")])
@pytest.mark.parametrize("T,N,K,r", SMALL)
def test_forward(T, N, K, r, dtype, dq, act):
    print(f"[gated] fwd {T} x {N} x {K} r {r} {dtype} dq {dq}", flush=True)
    Case(T, N, K, r, dtype, dq, act).check_fwd()


@pytest.mark.parametrize("dtype,dq,act", [("bf16", True, "silu"), ("bf16", False, "gelu_tanh"),
                                          ("fp16", True, "gelu_tanh"), ("fp16", False, "silu")])
@pytest.mark.parametrize("T,N,K,r", SMALL)
def test_backward(T, N, K, r, dtype, dq, act):
    print(f"[gated] bwd {T} x {N} x {K} r {r} {dtype} dq {dq}", flush=True)
    Case(T, N, K, r, dtype, dq, act).check_bwd()


# once-per-call dequantisation; split tiles (a last round at most half full) of
# either path and direction, with a reduction that ends inside a step
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K,r", [(2048, 256, 128, 16), (2300, 304, 320, 128),
                                     (1100, 6784, 1024, 16), (2100, 3712, 1024, 64)])
def test_forward_many_tokens(T, N, K, r, dtype):
    print(f"[gated] fwd {T} x {N} x {K} r {r} {dtype}", flush=True)
    Case(T, N, K, r, dtype).check_fwd()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K,r", [(2048, 256, 128, 16), (2300, 304, 320, 128),
                                     (1100, 528, 13568, 16), (2100, 592, 7424, 64)])
def test_backward_many_tokens(T, N, K, r, dtype):
    print(f"[gated] bwd {T} x {N} x {K} r {r} {dtype}", flush=True)
    Case(T, N, K, r, dtype).check_bwd()

"""Every form of the gated block's kernels: tiles of either size, whole and split
in two and more, weights decoded in LDS and once per call, reductions of whole
steps and with a rest, the streaming forward's splits; the form each size takes
is asserted without a GPU in test_gated_plans_cpu.py."""
import pytest

from test_gpu_gated import Case

pytestmark = pytest.mark.gpu

FWD_FORMS = [(1, 48, 1024, 16), (16, 1008, 4096, 48), (3, 64, 2048, 64), (5, 272, 4288, 96),
             (1, 32, 4544, 128), (20, 528, 4288, 16), (75, 16, 576, 16), (400, 9600, 64, 64),
             (269, 11952, 64, 16), (158, 9824, 3904, 64), (2804, 1952, 64, 64),
             (3195, 1568, 64, 96), (2861, 2864, 1024, 16)]
BWD_FORMS = [(1, 256, 64, 64), (1, 224, 64, 96), (1833, 64, 5120, 96), (420, 16, 17024, 96),
             (174, 2496, 18176, 96), (138, 2416, 16512, 96), (3176, 64, 3136, 16),
             (3871, 16, 2624, 96), (2267, 640, 9088, 16), (2187, 672, 7552, 64)]
FORMATS = [("bf16", True, "silu"), ("bf16", False, "gelu_tanh"), ("fp16", True, "gelu_tanh"),
           ("fp16", False, "silu")]


@pytest.mark.parametrize("dtype,dq,act", FORMATS)
@pytest.mark.parametrize("T,N,K,r", FWD_FORMS)
def test_forward_form(T, N, K, r, dtype, dq, act):
    print(f"[gated] fwd {T} x {N} x {K} r {r} {dtype} dq {dq}", flush=True)
    Case(T, N, K, r, dtype, dq, act).check_fwd()


@pytest.mark.parametrize("dtype,dq,act", FORMATS)
@pytest.mark.parametrize("T,N,K,r", BWD_FORMS)
def test_backward_form(T, N, K, r, dtype, dq, act):
    print(f"[gated] bwd {T} x {N} x {K} r {r} {dtype} dq {dq}", flush=True)
    Case(T, N, K, r, dtype, dq, act).check_bwd()

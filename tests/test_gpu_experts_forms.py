"""Every form of the expert-grouped kernels against the 64-bit formulas: each
tile and streaming form in either 16-bit type, with and without double
quantisation, the backward with a reduction that ends inside a step or not.
Which form a case takes is asserted without a GPU in test_plans_cpu.py."""
import pytest

from test_gpu_experts import BF, HF, check, make

pytestmark = pytest.mark.gpu

COUNTS = {"stream_16": [5, 0, 3, 9], "stream_32": [20, 0, 33, 9],
          "tiles_128": [90, 0, 200, 131, 7], "tiles_256": [300, 0, 129, 512] + [257] * 21}
# N, K, r of each; N % 64 is not 0 or is, which the backward tells apart
SHAPES = {"stream_16": [(272, 576, 48)], "stream_32": [(272, 576, 16)],
          "tiles_128": [(272, 576, 32), (320, 576, 80)],
          "tiles_256": [(1040, 1088, 96), (1088, 1088, 64)]}
FORM_CASES = [(f"{form}-{N}-{'fp16' if dt == HF else 'bf16'}-{'dq' if dq else 'constants'}",
               COUNTS[form], N, K, r, dt, 1, 2, dq)
              for form in COUNTS for N, K, r in SHAPES[form] for dt in (BF, HF)
              for dq in (True, False)]
# dA and dB from several parts of an expert's rows, the terms of G in fp16 or
# bf16; the last round's tiles split, in 128- and in 256-row tiles
FORM_CASES += [("rows_in_parts", [1500, 700], 272, 576, 16, HF, 0, 3, True),
               ("rows_in_parts_bf16", [1500, 700], 272, 576, 80, BF, 2, 0, False),
               ("split_of_128", [130, 300, 257], 2112, 1088, 64, HF, 0, 0, True),
               ("split_of_256", [300] * 20, 2112, 2048, 16, HF, 0, 0, True),
               ("split_of_256_bf16", [300] * 20, 2112, 2048, 32, BF, 0, 1, False)]


@pytest.mark.parametrize("case", FORM_CASES, ids=[c[0] for c in FORM_CASES])
def test_form(case):
    name, counts, N, K, r, dtype, lead, tail, dq = case
    print(f"[experts] {name}", flush=True)
    check(make(counts, N, K, r, dtype, lead, tail, dq), dtype, r)

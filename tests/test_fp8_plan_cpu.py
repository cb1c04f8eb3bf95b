"""The 8-bit floating point plan has no step at a number of bytes of the weight, and
splits and quantises as its comment says."""
import shutil

import pytest

import gated_plans as plans

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("cols", [4096, 5120, 8192, 11008, 16384, 22016])
def test_one_row_more_changes_nothing(gated, cols):
    """Where a weight passes 10^8 bytes, within one row of tiles."""
    rows = 10 ** 8 // cols // (2 if gated else 1)
    assert rows % 64
    for T in (1, 7, 12, 24, 40, 64, 80, 100, 150, 211, 317, 512):
        for x16 in (False, True):
            low, high = plans.fp8_plans([(T, rows, cols), (T, rows + 1, cols)], gated, x16)
            assert low == high, (T, rows, cols, x16)


def test_weights_past_the_cache_are_split():
    """From memory, us: 7 x 14336 x 8192 27 in 4 parts, 40 unsplit; 80 x 8192 x 22016
    49.5 in 4, 62 in 2; 12 x 12210 x 8192 25 and 39."""
    sizes = [(7, 14336, 8192), (80, 8192, 22016), (12, 12210, 8192), (24, 14336, 8192)]
    assert all(s >= 3 for _, s in plans.fp8_plans(sizes, False, False)), plans.fp8_plans(sizes, False, False)


def test_few_tokens_are_quantised_within_the_call():
    """Where all workgroups together quantise at most 2^24 codes."""
    near = [(1, 4096, 4096), (1, 28672, 8192), (2, 32000, 4096), (8, 16384, 1024), (1, 22016, 8192)]
    far = [(4, 65536, 2048), (8, 100000, 1024), (3, 4096, 4096)]
    assert all(p == "fused" for p, _ in plans.fp8_plans(near, False, True))
    assert all(p != "fused" for p, _ in plans.fp8_plans(far, False, True))

"""The sizes of the GPU tests take every form of the 8-bit and the expert-grouped
kernels: a change of the plans that leaves one untested fails here."""
import itertools
import shutil

import pytest

import plans
from test_gpu_experts import CASES, HF
from test_gpu_experts_forms import FORM_CASES
from test_gpu_int8 import SIZES
from test_gpu_int8_forms import FORM_SIZES

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

TILES = {"64x128": (64, 128), "128x128": (128, 128), "128x256": (128, 256), "256x256": (256, 256)}


def test_int8_sizes_take_every_kernel():
    sizes = SIZES + FORM_SIZES
    taken = dict(zip(sizes, plans.int8_plans(sizes, True)))
    for tile, split in itertools.product(TILES, (False, True)):
        tm, tn = TILES[tile]
        these = [s for s, (p, n) in taken.items() if p == tile and (n > 1) == split]
        assert these, (tile, split)
        # ragged in tokens, outputs and the last step; outputs that no 8- or
        # 16-byte store takes whole
        assert any(t % tm and n % tn and k % 128 for t, n, k in these), (tile, split)
        assert any(n % 4 for t, n, k in these), (tile, split)
    streamed = [t for (t, n, k), (p, _) in taken.items() if p == "skinny"]
    for lo, hi in ((1, 16), (17, 32), (33, 64)):
        assert any(lo <= t <= hi for t in streamed), (lo, hi)


def test_long_reductions_of_large_weights_are_split():
    """640 x 8192 x 22016: 128 us in two parts, 154 unsplit; 211 x 8192 x 14336
    44 against 52.  The same tokens on smaller weights stay unsplit."""
    split = plans.int8_plans([(640, 8192, 22016), (211, 8192, 14336), (500, 5504, 22016)], True)
    whole = plans.int8_plans([(640, 4096, 11008), (640, 22016, 8192), (8192, 11008, 4096)], True)
    assert all(n > 1 for _, n in split) and all(n == 1 for _, n in whole), (split, whole)


def test_int8_linear_sizes_take_every_way_of_quantising():
    """The sizes of test_linear_is_quantize_then_product: within the streaming
    kernel, by a launch before it, before tiles whole and split."""
    sizes = list(itertools.product([1, 2, 5, 16, 40, 64, 65, 150, 700],
                                   [(272, 1040), (1024, 4096), (48, 22016)]))
    taken = plans.int8_plans([(t, n, k) for t, (n, k) in sizes], False)
    paths = {p for p, _ in taken}
    assert {"fused", "skinny"} <= paths and len(paths) >= 3
    assert any(s > 1 for _, s in taken) and any(s == 1 and p in TILES for p, s in taken)


def _grouped(bwd):
    cases = [(c[1], c[2], c[3], c[4], c[5] == HF, c[8], sum(c[1]) + c[6] + c[7])
             for c in CASES + FORM_CASES if sum(c[1]) + c[6] + c[7] > 0]
    return list(zip(cases, plans.grouped_plans(cases, bwd)))


FORMATS = list(itertools.product((False, True), (False, True)))   # fp16, double quantisation


def test_grouped_cases_take_every_forward():
    got = _grouped(False)
    for f16, dq in FORMATS:
        mine = [p for c, p in got if (c[4], c[5]) == (f16, dq)]
        for rows in (16, 32):
            assert any(p["skinny"] == rows for p in mine), (f16, dq, rows)
        for mi in (2, 4):
            assert any(not p["skinny"] and p["mi"] == mi for p in mine), (f16, dq, mi)
    for mi in (2, 4):
        assert any(not p["skinny"] and p["mi"] == mi and p["parts"] > 1 for _, p in got), mi
    assert any(p["skinny"] and p["s_gemv"] > 1 for _, p in got)


def test_grouped_cases_take_every_backward():
    got = _grouped(True)
    for f16, dq, mi, tail in itertools.product((False, True), (False, True), (2, 4), (False, True)):
        assert any((c[4], c[5]) == (f16, dq) and p["mi"] == mi and (c[1] % 64 != 0) == tail
                   for c, p in got), (f16, dq, mi, tail)
    for f16 in (False, True):
        assert any(p["s_grad"] > 1 and c[4] == f16 for c, p in got), f16
        for mi in (2, 4):
            assert any(p["mi"] == mi and p["parts"] > 1 and c[4] == f16 for c, p in got), (f16, mi)
    # every rank's kernels of the projection and of the gradients
    assert {c[3] // 16 for c, _ in got} == set(range(1, 9))

"""The sizes of the GPU tests take every form of the 8-bit floating point and the
gated kernels: a change of the plans that leaves one untested fails here."""
import itertools
import shutil

import pytest

import gated_plans as plans
from test_gpu_fp8 import SIZES
from test_gpu_fp8_forms import FORM_SIZES, GATED_FORM_SIZES
from test_gpu_gated import SMALL
from test_gpu_gated_forms import BWD_FORMS, FWD_FORMS

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

TILES = {"64x128": (64, 128), "128x128": (128, 128), "128x256": (128, 256), "256x256": (256, 256)}


@pytest.mark.parametrize("gated", [False, True])
def test_fp8_sizes_take_every_kernel(gated):
    sizes = SIZES + (GATED_FORM_SIZES if gated else FORM_SIZES)
    taken = dict(zip(sizes, plans.fp8_plans(sizes, gated, False)))
    for tile, split in itertools.product(TILES, (False, True)):
        tm, tn = TILES[tile]
        these = [s for s, (p, n) in taken.items() if p == tile and (n > 1) == split]
        # ragged in tokens, outputs and the last step; outputs that no 8- or
        # 16-byte store takes whole
        assert any(t % tm and n % tn and k % 128 for t, n, k in these), (tile, split)
        assert any(n % 4 for t, n, k in these), (tile, split)
    streamed = [t for (t, n, k), (p, _) in taken.items() if p == "skinny"]
    for lo, hi in ((1, 16), (17, 32)):
        assert any(lo <= t <= hi for t in streamed), (lo, hi)
    quantised = {p for p, _ in plans.fp8_plans(sizes, gated, True)}
    assert {"fused", "skinny", "64x128"} <= quantised, quantised


def test_gated_sizes_take_every_forward():
    sizes = SMALL + FWD_FORMS
    got = list(zip(sizes, plans.gated(sizes, False)))
    for s in (1, 2, 4, 8):
        assert any(p["s_gemv"] == s for _, p in got), s
    for lo, hi in ((1, 4), (5, 16), (17, 32), (33, 64)):
        assert any(lo <= c[0] <= hi and p["s_gemv"] for c, p in got), (lo, hi)
    tiled = [(c, p) for c, p in got if not p["s_gemv"]]
    for split in (False, True):
        for mi in (2, 4):
            assert any(p["mi"] == mi and not p["pre_dq"] and (p["split"] > 0) == split
                       for _, p in tiled), (mi, split)
        assert any(p["pre_dq"] and (p["split"] > 0) == split for _, p in tiled), split
    assert any(p["parts"] > 2 for _, p in tiled)


def test_gated_sizes_take_every_backward():
    sizes = SMALL + BWD_FORMS
    got = list(zip(sizes, plans.gated(sizes, True)))
    for split, tail in itertools.product((False, True), (False, True)):
        these = [p for c, p in got if (p["split"] > 0) == split and (c[1] % 64 != 0) == tail]
        for mi in (2, 4):
            assert any(p["mi"] == mi and not p["pre_dq"] for p in these), (mi, split, tail)
        assert any(p["pre_dq"] for p in these), (split, tail)
    assert any(p["parts"] > 2 for _, p in got)
    assert any(p["s_grad"] > 1 for _, p in got) and any(p["s_proj"] > 1 for _, p in got)
    assert {c[3] // 16 for c in sizes} == set(range(1, 9))   # every rank's kernels

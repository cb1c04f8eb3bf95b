"""The tiled products in 8-bit floating point wait for their LDS loads by count
(s_waitcnt vmcnt(N) before a step's barrier), so every step has to issue exactly
the vector-memory loads that the count was made from, also the last steps, whose
loads nobody uses.  fp8.hip is compiled for gfx950 to assembly and the loads
between the barriers of every kernel are counted."""
import os
import re
import shutil
import subprocess

import pytest

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")

KERNEL = re.compile(r"^(_ZN5qlora\w*15fp8_gemm_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", re.M | re.S)
TILE = re.compile(r"F8TileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)EEELb([01])ELb([01])ELb([01])E")


def test_every_step_issues_the_loads_its_wait_counts(tmp_path):
    from bit_nf4_quantized_06_amd import build as B
    out = tmp_path / "fp8.s"
    subprocess.run([HIPCC] + B.hipcc_flags() + ["--cuda-device-only", "-S", "-o", str(out),
                                                os.path.join(B.CSRC, "fp8.hip")],
                   check=True, capture_output=True, timeout=600)
    kernels = KERNEL.findall(out.read_text())
    # 4 tiles, two types, whole or split, linear or gated
    assert len(kernels) == 32
    for name, body in kernels:
        mi, wm, wn, sw, sx, _, _, gated = map(int, TILE.search(name).groups())
        waves = wm * wn
        lx, lw = 16 * mi * wm // 8 // waves, 64 * wn // 8 // waves
        scales = (mi + 3) // 4 + (2 if gated else 1)
        keep = (sx - 2) * (lx + lw + scales) + (0 if sw == sx else lw)
        lines = [l.strip() for l in body.splitlines()]
        at = [i for i, l in enumerate(lines) if l.startswith("s_barrier")]
        unroll = sw if sw == sx else sw * sx
        # the prologue's, a group's, the last steps' (and the epilogue's)
        assert len(at) >= 1 + unroll + unroll - 1, name
        steps = at[:2 * unroll]
        for i in steps:
            wait = next(l for l in reversed(lines[:i]) if "vmcnt" in l)
            assert int(re.search(r"vmcnt\((\d+)\)", wait).group(1)) <= keep, (name, wait)
        for k, (a, b) in enumerate(zip(steps, steps[1:])):
            # from the barrier before a step's last products to the next step's;
            # past the loop's (both sides of a branch may hold the same loads)
            n = sum(l.startswith("buffer_load") for l in lines[a:b])
            if k < unroll:
                assert n == lx + lw + scales, (name, k, n, lx, lw, scales)
            else:
                assert n >= lx + lw + scales, (name, k, n, lx, lw, scales)

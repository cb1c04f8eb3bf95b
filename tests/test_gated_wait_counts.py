"""The gated block's backward waits for the loads of B into LDS by count (s_waitcnt
vmcnt(20) before an iteration's barrier: 8 stores and 12 loads are newer), so
every iteration has to issue exactly those, the last ones too, whose loads nobody
uses.  gated.hip is compiled for gfx950 to assembly and they are counted."""
import os
import re
import shutil
import subprocess

import pytest

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")

KERNEL = re.compile(r"^(_ZN5qlora16gated_bwd_kernelILi(\d)\w+):[^\n]*\n(.*?)^\.Lfunc_end", re.M | re.S)


def test_every_iteration_issues_what_its_wait_counts(tmp_path):
    from bit_nf4_quantized_06_amd import build as B
    out = tmp_path / "gated.s"
    subprocess.run([HIPCC] + B.hipcc_flags() + ["--cuda-device-only", "-S", "-o", str(out),
                                                os.path.join(B.CSRC, "gated.hip")],
                   check=True, capture_output=True, timeout=600)
    kernels = KERNEL.findall(out.read_text())
    assert len(kernels) == 32        # ranks, types, activations
    for name, nj, body in kernels:
        lines = [l.strip() for l in body.splitlines()]
        at = [i for i, l in enumerate(lines) if l.startswith("s_barrier")]
        assert len(at) == 3, name    # the loop's two iterations and the odd one
        for i in at:
            wait = next(l for l in reversed(lines[:i]) if "vmcnt" in l)
            assert int(re.search(r"vmcnt\((\d+)\)", wait).group(1)) <= 20, (name, wait)
            end = next(k for k in range(i + 1, len(lines))
                       if lines[k].startswith(("s_barrier", "s_cbranch", ".LBB")))
            ops = [l for l in lines[i:end] if l.startswith("buffer_")]
            dma = [k for k, l in enumerate(ops) if l.endswith("lds")]
            assert dma == list(range(int(nj))), (name, dma)   # B's first
            new = ops[int(nj):]
            assert sum(l.startswith("buffer_store") for l in new) == 8, name
            assert sum(l.startswith("buffer_load") for l in new) == 12, name

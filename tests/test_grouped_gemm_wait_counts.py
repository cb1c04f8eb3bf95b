"""The expert-grouped GEMM's wait for its seed keeps no more vector-memory
operations outstanding than were issued after the seed's loads.

As for the dense kernels (test_gemm_wait_counts.py): the first wait after the
8 DMAs of the adapter's operands may leave outstanding only the loads of steps
0 and 1.  A load that the compiler drops would make the count one too large,
and the seed would be read while still in flight; one more than counted
(offsets, scales) only makes the wait longer.
"""
import re

import pytest

from test_gemm_wait_counts import LOAD, VMCNT, gemm_asm, pytestmark  # noqa: F401

KERNEL = re.compile(r"^(_ZN5qlora19grouped_gemm_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", re.M | re.S)


def test_every_grouped_kernel_waits_for_its_seed_loads(gemm_asm):  # noqa: F811
    kernels = KERNEL.findall(gemm_asm)
    # <backward, double quantisation, fp16, tile, ragged end>: 2 x 2 forwards and
    # 2 x 2 x 2 backwards in two tiles
    assert len(kernels) == 24, [k for k, _ in kernels]
    for name, body in kernels:
        lines = body.splitlines()
        first = next(i for i, l in enumerate(lines) if LOAD.match(l) and l.rstrip().endswith(" lds"))
        waits = [i for i in range(first, len(lines)) if VMCNT.search(lines[i])]
        kept = int(VMCNT.search(lines[waits[0]]).group(1))
        issued = sum(1 for l in lines[first:waits[0]] if LOAD.match(l))
        assert issued >= 8 + kept, f"{name}: {issued} loads before a wait keeping {kept}"

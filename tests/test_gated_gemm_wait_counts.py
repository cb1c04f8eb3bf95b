"""The gated GEMM's wait for its adapters' operands keeps exactly the loads issued
after them outstanding, and each step's wait exactly the loads issued in the step.

As for the dense kernels (test_gemm_wait_counts.py): a load that the compiler
drops, or moves across a wait, would make a count too large, and a stage would be
read while still in flight."""
import re

from test_gemm_wait_counts import VMCNT, gemm_asm, pytestmark  # noqa: F401

KERNEL = re.compile(r"^(_ZN5qlora17gated_gemm_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", re.M | re.S)
# <backward, double quantisation, fp16, once-per-call dequantisation, ragged end, tile>
PARAMS = re.compile(r"ILb([01])ELb([01])ELb([01])ELb([01])ELb([01])ELi(\d)E")


def instructions(body):
    return [l.strip() for l in body.splitlines()]


def loads(lines):
    return sum(l.startswith("buffer_load") for l in lines)


def branches(line):
    return line.startswith((".LBB", "s_cbranch", "s_branch", "s_setpc"))


def waits(lines, lo=0):
    """(index, count) of every wait for vector memory"""
    return [(i, int(VMCNT.search(l).group(1))) for i, l in enumerate(lines) if i >= lo and VMCNT.search(l)]


def test_every_gated_kernel_waits_for_its_adapters_and_its_steps(gemm_asm):  # noqa: F811
    kernels = KERNEL.findall(gemm_asm)
    # forwards: 2 x 2 formats in two tiles, 2 types dequantised once; backwards the
    # same with and without a ragged end
    assert len(kernels) == 30, [k for k, _ in kernels]
    for name, body in kernels:
        _, dq, _, once, _, _ = map(int, PARAMS.search(name).groups())
        prologue, step = (8, 8) if once else ((14, 7) if dq else (12, 6))
        lines = instructions(body)
        # the adapters' first operands: 8 DMAs, 4 more above rank 32 (a block of its
        # own), then the stages' first loads up to the wait
        first = next(i for i, l in enumerate(lines) if l.startswith("buffer_load"))
        wait, kept = waits(lines, first)[0]
        assert kept == prologue, (name, kept)
        blocks = [[]]
        for l in lines[first:wait]:
            if branches(l):
                blocks.append([])
            else:
                blocks[-1].append(l)
        blocks = [b for b in blocks if loads(b)]
        assert [loads(b) for b in blocks] == [8, 4, prologue], (name, list(map(loads, blocks)))
        assert all(l.endswith(" lds") for b in blocks[:2] for l in b if l.startswith("buffer_load"))
        # steps: between two barriers of one basic block
        at = [i for i, l in enumerate(lines) if l.startswith("s_barrier")]
        pairs = 0
        for a, b in zip(at, at[1:]):
            between = lines[a + 1:b]
            if any(map(branches, between)) or loads(between) == 0:
                continue
            kept = [c for _, c in waits(between)]
            assert loads(between) == step and kept and kept[-1] <= step, (name, loads(between), kept)
            pairs += 1
        assert pairs >= 5, (name, pairs)      # six steps a turn of the loop

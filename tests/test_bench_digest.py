"""The digest under which bench.py takes a committed traffic profile covers the
kernel file and every header it includes, so an edit of any of them leaves the
profile behind."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "bit_nf4_quantized_06_amd", "csrc")


@pytest.mark.parametrize("kernel,some", [
    ("gemm.hip", {"device_common.h", "gemm_common.h", "group.h", "grouped.h", "grouped_kernels.h",
                  "kernels.h", "abi_internal.h"}),
    ("gemv.hip", {"device_common.h", "group.h", "grouped.h", "grouped_kernels.h", "kernels.h",
                  "abi_internal.h"})])
def test_every_included_header_is_in_the_digest(kernel, some, tmp_path, monkeypatch):
    names = bench.kernel_sources(kernel)
    assert names[0] == kernel and some <= set(names) and len(names) == len(set(names))
    # nothing of the folder that one of them includes is left out
    for n in names:
        for line in open(os.path.join(CSRC, n)):
            if line.lstrip().startswith("#include") and '"' in line:
                inc = line.split('"')[1]
                assert inc in names or not os.path.exists(os.path.join(CSRC, inc)), (n, inc)
    copy = tmp_path / "bit_nf4_quantized_06_amd" / "csrc"
    shutil.copytree(CSRC, copy)
    before = bench.source_digest(kernel)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.source_digest(kernel) == before
    seen = {before}
    for n in names:
        with open(copy / n, "a") as f:
            f.write("// edited\n")
        now = bench.source_digest(kernel)
        assert now not in seen, n
        seen.add(now)
    with open(copy / "merge.hip", "a") as f:
        f.write("// another kernel\n")
    assert bench.source_digest(kernel) == now

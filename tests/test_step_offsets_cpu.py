"""Addresses of the tiled GEMMs' loads that run past a reduction's or a part's end:
no lane's and step's offset are out of range at the same time, where their 32-bit
sum would be an address in the tensor again."""
import os
import shutil
import subprocess

import pytest

from bit_nf4_quantized_06_amd import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def test_no_offset_wraps(tmp_path):
    _lib.load()
    exe = tmp_path / "step_offsets_check"
    tlib = build._torch_lib_dir()
    subprocess.run(["g++", *build.host_flags(), os.path.join(ROOT, "tests", "c", "step_offsets_check.cpp"),
                    "-o", str(exe), build.LIB_PATH, f"-L{tlib}", "-l:libamdhip64.so",
                    f"-Wl,-rpath,{tlib}:{build.PKG}"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
    looked, past_end_tails = map(int, out.stdout.split())
    assert looked > 10 ** 6 and past_end_tails > 100

"""How the 8-bit floating point and the gated entry points run given sizes, from
the library's own plan functions (host code, no GPU)."""
import os
import subprocess
import tempfile
from functools import lru_cache

from bit_nf4_quantized_06_amd import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FP8_PATHS = ["fused", "skinny", "64x128", "128x128", "128x256", "256x256"]


@lru_cache(maxsize=1)
def _exe():
    _lib.load()                       # built if it is not there yet
    exe = os.path.join(tempfile.mkdtemp(), "gated_plan_check")
    tlib = build._torch_lib_dir()
    subprocess.run(["g++", *build.host_flags(),
                    os.path.join(ROOT, "tests", "c", "gated_plan_check.cpp"), "-o", exe,
                    build.LIB_PATH, f"-L{tlib}", "-l:libamdhip64.so",
                    f"-Wl,-rpath,{tlib}:{build.PKG}"], check=True)
    return exe


def _ask(lines):
    out = subprocess.run([_exe()], input="\n".join(lines) + "\n", capture_output=True, text=True,
                         timeout=60, check=True).stdout.splitlines()
    assert len(out) == len(lines), out
    return [[int(v) for v in l.split()] for l in out]


def fp8_plans(sizes, gated, x16):
    """(path, splits) of each (T, rows, cols)."""
    return [(FP8_PATHS[p], s) for p, s in
            _ask([f"fp8 {t} {2 * n if gated else n} {k} {int(x16)}" for t, n, k in sizes])]


def gated(sizes, bwd):
    """A dict for each (T, rows, cols, r)."""
    names = ("s_gemv", "mi", "pre_dq", "split", "parts", "s_proj", "s_grad")
    return [dict(zip(names, v)) for v in
            _ask([f"gated {t} {n} {k} {r} {int(bwd)}" for t, n, k, r in sizes])]

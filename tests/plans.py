"""How the 8-bit and the expert-grouped entry points run given sizes, from the
library's own plan functions (host code, no GPU)."""
import os
import subprocess
import tempfile
from functools import lru_cache

from bit_nf4_quantized_06_amd import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INT8_PATHS = ["fused", "skinny", "64x128", "128x128", "128x256", "256x256"]


@lru_cache(maxsize=1)
def _exe():
    _lib.load()                       # built if it is not there yet
    exe = os.path.join(tempfile.mkdtemp(), "plan_check")
    tlib = build._torch_lib_dir()
    subprocess.run(["g++", *build.host_flags(), os.path.join(ROOT, "tests", "c", "plan_check.cpp"),
                    "-o", exe, build.LIB_PATH, f"-L{tlib}", "-l:libamdhip64.so",
                    f"-Wl,-rpath,{tlib}:{build.PKG}"], check=True)
    return exe


def _ask(lines):
    out = subprocess.run([_exe()], input="\n".join(lines) + "\n", capture_output=True, text=True,
                         timeout=60, check=True).stdout.splitlines()
    assert len(out) == len(lines), out
    return [[int(v) for v in l.split()] for l in out]


def int8_plans(sizes, given):
    """(path, splits) of each (T, rows, cols)."""
    return [(INT8_PATHS[p], s) for p, s in
            _ask([f"int8 {t} {n} {k} {int(given)}" for t, n, k in sizes])]


def grouped_plans(cases, bwd):
    """A dict for each (counts, rows, cols, r, fp16, double quantisation, T)."""
    lines = [f"group {n} {k} {r} {int(dq)} {int(f16)} {int(bwd)} {T} " + " ".join(map(str, counts))
             for counts, n, k, r, f16, dq, T in cases]
    names = ("skinny", "mi", "s_gemv", "s_proj", "s_grad", "parts")
    return [dict(zip(names, v)) for v in _ask(lines)]

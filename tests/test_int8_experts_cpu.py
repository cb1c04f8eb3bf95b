"""The 8-bit and the expert-grouped linear layer without a GPU: the headers'
functions are exported and bound, bad arguments are refused before a device
is touched, the code arithmetic is exact, and the reference formulas of the
grouped layer agree with differences."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import bit_nf4_quantized_06_amd as q
from bit_nf4_quantized_06_amd import _lib
from experts_ref import grouped_backward, grouped_forward
from test_kernel_arith_host import fma32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000          # aligned non-NULL "device" address; never dereferenced
MISALIGNED = 0x10008
NULL, SHAPE, ALIGN, WORKSPACE, FORMAT = 1, 2, 3, 4, 7
NO_DEVICE = (5, 6)      # what a call that passes every check meets here


@pytest.mark.parametrize("header,count", [("qlora_int8.h", 4), ("qlora_experts.h", 3)])
def test_header_functions_exported_and_bound(header, count):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(qlora_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == count, names
    lib = _lib.load()
    for name in names:
        assert hasattr(lib, name) and name in _lib.SIGNATURES, name
        assert hasattr(q, name), name


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("header", ["qlora_int8.h", "qlora_experts.h"])
def test_headers_compile_as_c99(header):
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    "-I", os.path.join(ROOT, "include"), "-x", "c", "-fsyntax-only", "-"],
                   input=f'#include "{header}"\nint main(void) {{ return 0; }}\n', text=True,
                   check=True)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_group_rows_stay_inside(tmp_path):
    exe = str(tmp_path / "group_rows")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "bit_nf4_quantized_06_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "group_rows_check.cpp"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


# --------------------------------------------------------------------------
# refusals of the C ABI
# --------------------------------------------------------------------------
def test_int8_quantize_refusals():
    f = _lib.load().qlora_int8_quantize
    assert f(FAKE, 0, 4, 64, FAKE, FAKE, None) in NO_DEVICE
    for t in (-1, 3):
        assert f(FAKE, t, 4, 64, FAKE, FAKE, None) == FORMAT
    for rows, cols in ((-1, 64), (4, 0), (4, 8), (4, 24), (4, 1 << 17), (1 << 22, 64)):
        assert f(FAKE, 0, rows, cols, FAKE, FAKE, None) == SHAPE, (rows, cols)
    for k in range(3):
        for bad, code in ((None, NULL), (MISALIGNED, ALIGN)):
            p = [FAKE] * 3
            p[k] = bad
            assert f(p[0], 0, 4, 64, p[1], p[2], None) == code
    assert f(None, 0, 0, 64, None, None, None) in NO_DEVICE      # no rows: nothing to do


@pytest.mark.parametrize("given", [True, False])
def test_int8_product_refusals(given):
    lib = _lib.load()

    def call(W=FAKE, ws_=FAKE, rows=128, cols=64, X=FAKE, xs=FAKE, T=70, cd=0, Y=FAKE, wk=FAKE,
             wb=1 << 40):
        if given:
            return lib.qlora_int8_matmul(W, ws_, rows, cols, X, xs, T, cd, Y, wk, wb, None)
        return lib.qlora_int8_linear_fwd(W, ws_, rows, cols, X, T, cd, Y, wk, wb, None)

    assert call() in NO_DEVICE
    assert call(cd=2) == FORMAT and call(cd=-1) == FORMAT
    for bad in (dict(rows=0), dict(rows=-16), dict(rows=1 << 22), dict(cols=0),
                dict(cols=24), dict(cols=1 << 17), dict(T=-1), dict(T=1 << 22),
                dict(T=1 << 20, rows=1 << 16)):
        assert call(**bad) == SHAPE, bad
    for name in ("W", "ws_", "X", "Y") + (("xs",) if given else ("wk",)):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: MISALIGNED}) == ALIGN, name
    need = lib.qlora_int8_workspace(70, 128, 64, int(given))
    if need:
        assert call(wb=need - 1) == WORKSPACE
        assert call(wb=need) in NO_DEVICE
    else:
        assert call(wk=None, wb=0) in NO_DEVICE
    assert call(T=0, X=None, xs=None, Y=None, wk=None, wb=0) in NO_DEVICE
    assert call(T=(1 << 16) - 1, rows=1 << 20, cols=16) in NO_DEVICE
    assert call(rows=1, T=1) in NO_DEVICE and call(rows=333, cols=1040) in NO_DEVICE


def test_int8_workspace_of_bad_arguments_is_zero():
    f = _lib.load().qlora_int8_workspace
    assert f(64, 128, 64, 0) >= 64 * 64 + 4 * 64
    for a in ((-1, 128, 64), (0, 128, 64), (64, 0, 64), (64, 128, 65), (64, 128, 1 << 18)):
        assert f(*a, 0) == 0 and f(*a, 1) == 0, a


def _stack(experts, rows, cols, qt=0, dq=1, f16=0):
    d = _lib.Nf4WeightDesc()
    assert _lib.load().qlora_nf4_weight_init_ex(ctypes.byref(d), experts * rows, cols, qt, dq,
                                                f16) == 0
    d.codes = d.absmax_code = d.absmax_scale = d.absmax_offset = FAKE
    return d


@pytest.mark.parametrize("bwd", [False, True])
def test_grouped_refusals(bwd):
    lib = _lib.load()

    def call(d=None, E=4, X=FAKE, dY=FAKE, T=200, off=FAKE, A=FAKE, B=FAKE, r=16, alpha=16.0,
             U=FAKE, out=FAKE, dA=FAKE, dB=FAKE, wk=FAKE, wb=1 << 40):
        d = ctypes.byref(d if d is not None else _stack(4, 128, 256))
        if bwd:
            return lib.qlora_grouped_linear_bwd(d, E, X, dY, T, off, A, B, r, alpha, U, out, dA,
                                                dB, wk, wb, None)
        return lib.qlora_grouped_linear_fwd(d, E, X, T, off, A, B, r, alpha, out, U, wk, wb, None)

    assert call() in NO_DEVICE
    for bad in (dict(E=0), dict(E=-4), dict(E=3), dict(E=64), dict(r=0), dict(r=8), dict(r=24),
                dict(r=144), dict(alpha=float("nan")), dict(alpha=float("inf")), dict(T=-1),
                dict(T=1 << 23), dict(E=1025, d=_stack(1025, 16, 64)),
                dict(E=1, d=_stack(1, (1 << 20) + 16, 64)), dict(E=1, d=_stack(1, 16, (1 << 20) + 64)),
                # the planes of G would pass 32-bit offsets
                dict(d=_stack(4, 16, 64), T=1 << 21, r=128)):
        assert call(**bad) == SHAPE, bad
    assert call(d=_stack(4, 128, 256, qt=1)) == FORMAT
    bad = _stack(4, 128, 256)
    bad.codes = None
    assert call(d=bad) == NULL
    names = ["X", "off", "A", "B", "out", "wk"] + (["dY", "U", "dA", "dB"] if bwd else [])
    for name in names:
        assert call(**{name: None}) == NULL, name
        assert call(**{name: MISALIGNED}) == ALIGN, name
    if not bwd:
        assert call(U=None) in NO_DEVICE and call(U=MISALIGNED) == ALIGN
    for T in (1, 200, 4000):
        need = lib.qlora_grouped_linear_workspace(T, 4, 128, 256, 16, 0, int(bwd))
        assert need > 0
        assert call(T=T, wb=need - 1) == WORKSPACE
        assert call(T=T, wb=need) in NO_DEVICE
    assert call(T=0, X=None, dY=None, U=None, wk=None, wb=0,
                **({} if bwd else {"out": None})) in NO_DEVICE


def test_grouped_workspace_of_bad_arguments_is_zero():
    f = _lib.load().qlora_grouped_linear_workspace
    for a in ((0, 4, 128, 256, 16, 0), (-1, 4, 128, 256, 16, 0), (9, 0, 128, 256, 16, 0),
              (9, 1025, 128, 256, 16, 0), (9, 4, 100, 256, 16, 0), (9, 4, 128, 100, 16, 0),
              (9, 4, 128, 256, 20, 0), (9, 4, 128, 256, 16, 2)):
        assert f(*a, 0) == 0 and f(*a, 1) == 0, a


# --------------------------------------------------------------------------
# refusals of the binding
# --------------------------------------------------------------------------
def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    x = torch.zeros(4, 64, dtype=bf)
    w = q.Int8Weight(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8))
    codes, xs = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="on a GPU"):
        q.qlora_int8_quantize(x)
    with pytest.raises(ValueError, match="on a GPU"):
        q.qlora_int8_linear_fwd(w, x)
    with pytest.raises(ValueError, match="on a GPU"):
        q.qlora_int8_matmul(w, codes, xs)
    with pytest.raises(TypeError):
        q.qlora_int8_quantize(x.to(torch.float64))
    with pytest.raises(TypeError):
        q.qlora_int8_linear_fwd(w, x.float())
    with pytest.raises(TypeError):
        q.qlora_int8_matmul(w, codes, xs, dtype=torch.float32)
    with pytest.raises(TypeError):
        q.qlora_int8_matmul(w, x, xs)
    with pytest.raises(TypeError):
        q.qlora_int8_linear_fwd(q.Int8Weight(w.codes.view(torch.uint8), w.scale), x)
    with pytest.raises(ValueError, match="shape"):
        q.qlora_int8_matmul(w, codes, xs[:3])
    with pytest.raises(ValueError, match="shape"):
        q.qlora_int8_linear_fwd(w, x[:, :32].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_int8_linear_fwd(w, torch.zeros(64, 4, dtype=bf).T)
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_int8_linear_fwd(w, x, Y=torch.zeros(8, 4, dtype=bf).T)


def test_grouped_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    E, N, K, r, T = 2, 32, 64, 16, 5
    w = q.NF4Weight(E * N, K, torch.zeros(E * N * K // 2, dtype=torch.uint8),
                    torch.zeros(E * N * K // 64, dtype=torch.uint8), torch.zeros(1), torch.zeros(1))
    good = dict(X=torch.zeros(T, K, dtype=bf), offsets=torch.zeros(E + 1, dtype=torch.int32),
                A=torch.zeros(E, r, K, dtype=bf), B=torch.zeros(E, N, r, dtype=bf))

    def fwd(**kw):
        a = {**good, **kw}
        return q.qlora_grouped_linear_fwd(w, a["X"], a["offsets"], a["A"], a["B"], 16.0)

    with pytest.raises(ValueError, match="on a GPU"):
        fwd()
    with pytest.raises(TypeError):
        fwd(offsets=torch.zeros(E + 1, dtype=torch.int64))
    with pytest.raises(ValueError):
        fwd(offsets=torch.zeros(E, dtype=torch.int32))
    with pytest.raises(TypeError):
        fwd(X=good["X"].half())
    with pytest.raises(ValueError):
        fwd(A=torch.zeros(3, r, K, dtype=bf))
    with pytest.raises(ValueError):
        fwd(A=torch.zeros(r, K, dtype=bf))
    with pytest.raises(ValueError):
        fwd(B=torch.zeros(E, r, N, dtype=bf))
    with pytest.raises(ValueError, match="on a GPU"):
        q.qlora_grouped_linear_bwd(w, good["X"], torch.zeros(T, N, dtype=bf), good["offsets"],
                                   good["A"], good["B"], 16.0, torch.zeros(T, r, dtype=bf))
    with pytest.raises(ValueError):
        q.qlora_grouped_linear_bwd(w, good["X"], torch.zeros(T, N, dtype=bf), good["offsets"],
                                   good["A"], good["B"], 16.0, torch.zeros(T, r + 16, dtype=bf))


# --------------------------------------------------------------------------
# arithmetic
# --------------------------------------------------------------------------
def test_code_rule_is_exact_next_to_every_border():
    """The kernel's code of x (rounded product with the rounded reciprocal,
    settled by the one-FMA remainder against s / 2) equals the nearest integer
    to the real quotient x / s, ties to even, for x at, one and two ulps
    around every border (k + 1/2) s.  The real comparison is done in integers:
    x = a 2^p, s = b 2^q."""
    rng = np.random.default_rng(3)
    F = np.float32
    s = np.concatenate([(0.5 + rng.random(4000)).astype(F),
                        np.exp2(rng.integers(-60, 60, 2000)).astype(F),
                        (rng.integers(1, 1 << 12, 2000) / 64).astype(F)])
    k = rng.integers(-127, 128, s.size)
    border = ((k + 0.5) * s.astype(np.float64)).astype(F)
    xs = [border]
    for toward in (np.inf, -np.inf):
        y = border
        for _ in range(2):
            y = np.nextafter(y, F(toward))
            xs.append(y)
    x, s = np.concatenate(xs), np.tile(s, len(xs))
    keep = np.abs(x.astype(np.float64)) <= 127.4 * s.astype(np.float64)
    x, s = x[keep], s[keep]
    # the kernel's steps
    r = np.rint(x * (F(1) / s)).astype(F)
    e = fma32(-r, s, x)
    h = F(0.5) * s
    ri = r.astype(np.int64)
    off = (np.abs(e) > h) | ((np.abs(e) == h) & (ri % 2 != 0))
    got = np.clip(np.where(off, ri + np.where(e < 0, -1, 1), ri), -127, 127)
    # the real quotient
    for i in range(x.size):
        xn, xd = float(x[i]).as_integer_ratio()
        sn, sd = float(s[i]).as_integer_ratio()
        num, den = xn * sd, xd * sn
        low = num // den
        twice = 2 * (num - low * den)
        want = low + (1 if twice > den or (twice == den and low % 2) else 0)
        assert got[i] == max(-127, min(127, want)), (x[i], s[i], got[i], want)


def test_reference_gradients_agree_with_differences():
    """dX, dA, dB of the 64-bit formulas against central differences (the
    layer is bilinear, so they agree to rounding)."""
    rng = np.random.default_rng(5)
    E, N, K, r, T, alpha = 3, 6, 5, 2, 7, 3.0
    off = [1, 4, 4, 6]
    W, A, B = (rng.standard_normal(n) for n in ((E, N, K), (E, r, K), (E, N, r)))
    X, dY = rng.standard_normal((T, K)), rng.standard_normal((T, N))
    _, U = grouped_forward(X, W, A, B, off, alpha)
    dX, dA, dB = grouped_backward(X, dY, W, A, B, off, alpha, U)
    rows = slice(off[0], off[-1])

    def loss(x, a, b):
        y, _ = grouped_forward(x, W, a, b, off, alpha)
        return float((y[rows] * dY[rows]).sum())

    for i, g in enumerate((dX, dA, dB)):
        args = [X, A, B]
        for idx in np.ndindex(g.shape):
            v = []
            for h in (1e-3, -1e-3):
                p = [a.copy() for a in args]
                p[i][idx] += h
                v.append(loss(*p))
            d = (v[0] - v[1]) / 2e-3
            if i == 0 and not off[0] <= idx[0] < off[-1]:
                assert d == 0.0
            else:
                assert abs(d - g[idx]) <= 1e-8 * (1 + abs(d)), (i, idx)

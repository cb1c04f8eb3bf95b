"""The layer in 8-bit floating point and the gated blocks without a GPU: the
headers' functions are exported and bound, bad arguments are refused before a
device is touched, and the reference formulas agree with another form."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import bit_nf4_quantized_06_amd as q
import fp8_ref as R
import gated_ref as G
from bit_nf4_quantized_06_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000          # aligned non-NULL "device" address; never dereferenced
MISALIGNED = 0x10008
NULL, SHAPE, ALIGN, WORKSPACE, FORMAT = 1, 2, 3, 4, 7
NO_DEVICE = (5, 6)      # what a call that passes every check meets here


@pytest.mark.parametrize("header,count", [("qlora_fp8.h", 7), ("qlora_gated.h", 3)])
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
@pytest.mark.parametrize("header", ["qlora_fp8.h", "qlora_gated.h"])
def test_headers_compile_as_c99(header):
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    "-I", os.path.join(ROOT, "include"), "-x", "c", "-fsyntax-only", "-"],
                   input=f'#include "{header}"\nint main(void) {{ return 0; }}\n', text=True,
                   check=True)


# --------------------------------------------------------------------------
# refusals of the C ABI
# --------------------------------------------------------------------------
@pytest.mark.parametrize("weight", [False, True])
def test_fp8_quantize_refusals(weight):
    lib = _lib.load()
    f = lib.qlora_fp8_quantize_weight if weight else lib.qlora_fp8_quantize
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
    none = f(None, 0, 0, 64, None, None, None)
    assert none == SHAPE if weight else none in NO_DEVICE


@pytest.mark.parametrize("kind", ["matmul", "linear", "gated"])
def test_fp8_product_refusals(kind):
    lib = _lib.load()

    def call(W=FAKE, ws_=FAKE, W2=FAKE, ws2=FAKE, rows=128, cols=64, X=FAKE, xs=FAKE, T=70, act=0,
             cd=0, Y=FAKE, wk=FAKE, wb=1 << 40):
        if kind == "matmul":
            return lib.qlora_fp8_matmul(W, ws_, rows, cols, X, xs, T, cd, Y, wk, wb, None)
        if kind == "linear":
            return lib.qlora_fp8_linear_fwd(W, ws_, rows, cols, X, T, cd, Y, wk, wb, None)
        return lib.qlora_fp8_gated_fwd(W, ws_, W2, ws2, rows, cols, X, T, act, cd, Y, wk, wb, None)

    assert call() in NO_DEVICE
    assert call(cd=2) == FORMAT and call(cd=-1) == FORMAT
    for bad in (dict(rows=0), dict(rows=-16), dict(rows=1 << 22), dict(cols=0),
                dict(cols=24), dict(cols=1 << 17), dict(T=-1), dict(T=1 << 22),
                dict(T=1 << 20, rows=1 << 16)):
        assert call(**bad) == SHAPE, bad
    names = ["W", "ws_", "X", "Y"] + {"matmul": ["xs"], "linear": ["wk"],
                                      "gated": ["wk", "W2", "ws2"]}[kind]
    for name in names:
        assert call(**{name: None}) == NULL, name
        assert call(**{name: MISALIGNED}) == ALIGN, name
    if kind == "gated":
        need = lib.qlora_fp8_gated_workspace(70, 128, 64)
        assert call(act=2) == FORMAT and call(act=-1) == FORMAT
        assert call(T=1 << 19, rows=1 << 16) == SHAPE        # 2 rows outputs a token
        assert call(act=1) in NO_DEVICE
    else:
        need = lib.qlora_fp8_workspace(70, 128, 64, int(kind == "matmul"))
    if need:
        assert call(wb=need - 1) == WORKSPACE
        assert call(wb=need) in NO_DEVICE
    else:
        assert call(wk=None, wb=0) in NO_DEVICE
    assert call(T=0, X=None, xs=None, Y=None, wk=None, wb=0) in NO_DEVICE
    assert call(rows=1, T=1) in NO_DEVICE and call(rows=333, cols=1040) in NO_DEVICE


def test_fp8_workspace_of_bad_arguments_is_zero():
    lib = _lib.load()
    assert lib.qlora_fp8_workspace(65, 128, 64, 0) >= 65 * 64 + 4 * 65
    assert lib.qlora_fp8_gated_workspace(65, 128, 64) >= 65 * 64 + 4 * 65
    for a in ((-1, 128, 64), (0, 128, 64), (64, 0, 64), (64, 128, 65), (64, 128, 1 << 18)):
        assert lib.qlora_fp8_workspace(*a, 0) == 0 and lib.qlora_fp8_workspace(*a, 1) == 0, a
        assert lib.qlora_fp8_gated_workspace(*a) == 0, a


def _weight(rows=128, cols=256, qt=0, dq=1, f16=0):
    d = _lib.Nf4WeightDesc()
    assert _lib.load().qlora_nf4_weight_init_ex(ctypes.byref(d), rows, cols, qt, dq, f16) == 0
    d.codes = d.absmax_code = d.absmax_scale = d.absmax_offset = FAKE
    return d


@pytest.mark.parametrize("T", [1, 64, 65, 2100])
@pytest.mark.parametrize("bwd", [False, True])
def test_gated_refusals(bwd, T):
    lib = _lib.load()

    def call(gate=None, up=None, X=FAKE, dH=FAKE, T=T, Ag=FAKE, Bg=FAKE, Au=FAKE, Bu=FAKE, r=16,
             alpha=16.0, act=0, Pg=FAKE, Pu=FAKE, Ug=FAKE, Uu=FAKE, out=FAKE, dAg=FAKE, dBg=FAKE,
             dAu=FAKE, dBu=FAKE, wk=FAKE, wb=1 << 40):
        gate = ctypes.byref(_weight() if gate is None else gate)
        up = ctypes.byref(_weight() if up is None else up)
        if bwd:
            return lib.qlora_gated_linear_bwd(gate, up, X, dH, T, Ag, Bg, Au, Bu, r, alpha, act,
                                              Pg, Pu, Ug, Uu, out, dAg, dBg, dAu, dBu, wk, wb, None)
        return lib.qlora_gated_linear_fwd(gate, up, X, T, Ag, Bg, Au, Bu, r, alpha, act, out, Pg,
                                          Pu, Ug, Uu, wk, wb, None)

    assert call() in NO_DEVICE and call(act=1) in NO_DEVICE
    for bad in (dict(r=0), dict(r=8), dict(r=24), dict(r=144), dict(alpha=float("nan")),
                dict(alpha=float("inf")), dict(T=-1), dict(T=1 << 23),
                dict(up=_weight(144)), dict(up=_weight(128, 320)), dict(gate=_weight(128, 192))):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(act=-1), dict(act=2), dict(gate=_weight(qt=1)), dict(up=_weight(qt=1)),
                dict(up=_weight(dq=0)), dict(up=_weight(f16=1))):
        assert call(**bad) == FORMAT, bad
    for side in ("gate", "up"):
        bad = _weight()
        bad.codes = None
        assert call(**{side: bad}) == NULL
    names = ["X", "Ag", "Bg", "Au", "Bu", "out", "wk", "Pg", "Pu", "Ug", "Uu"]
    names += ["dH", "dAg", "dBg", "dAu", "dBu"] if bwd else []
    for name in names:
        assert call(**{name: None}) == NULL, name
        assert call(**{name: MISALIGNED}) == ALIGN, name
    if not bwd:        # what the backward needs: all of it or nothing
        assert call(Pg=None, Pu=None, Ug=None, Uu=None) in NO_DEVICE
    need = lib.qlora_gated_linear_workspace(T, 128, 256, 16, int(bwd))
    assert need > 0
    assert call(wb=need - 1) == WORKSPACE and call(wb=need) in NO_DEVICE
    assert call(T=0, X=None, dH=None, Pg=None, Pu=None, Ug=None, Uu=None, out=None, wk=None,
                wb=0) in NO_DEVICE


def test_gated_workspace_of_bad_arguments_is_zero():
    f = _lib.load().qlora_gated_linear_workspace
    for a in ((-1, 128, 256, 16), (0, 128, 256, 16), (70, 8, 256, 16), (70, 128, 100, 16),
              (70, 128, 256, 24), (70, 128, 256, 144), (1 << 23, 128, 256, 16)):
        assert f(*a, 0) == 0 and f(*a, 1) == 0, a


# --------------------------------------------------------------------------
# the binding's own checks (CPU tensors: nothing reaches the library's kernels)
# --------------------------------------------------------------------------
def _fp8(rows, cols):
    return q.Fp8Weight(torch.zeros(rows, cols).to(torch.float8_e4m3fn),
                       torch.ones(-(-rows // 128), -(-cols // 128)))


def test_fp8_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = _fp8(128, 64)
    with pytest.raises(TypeError):
        q.qlora_fp8_quantize(x.to(torch.float64))
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize(torch.zeros(64, 4, dtype=torch.bfloat16).T)
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize(torch.zeros(2, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize(x)                         # not on a GPU
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize(x, scale=torch.zeros(4, 1))
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize_weight(x, scale=torch.zeros(1, 4))
    with pytest.raises(TypeError):
        q.qlora_fp8_linear_fwd(w, x.float())
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(w, torch.zeros(4, 80, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(q.Fp8Weight(w.codes, torch.ones(1, 2)), x)
    with pytest.raises(TypeError):
        q.qlora_fp8_linear_fwd(q.Fp8Weight(w.codes.view(torch.int8), w.scale), x)
    with pytest.raises(TypeError):
        q.qlora_fp8_matmul(w, x, torch.ones(1, 4))
    with pytest.raises(ValueError):
        q.qlora_fp8_matmul(w, x.to(torch.float8_e4m3fn), torch.ones(4, 1))
    with pytest.raises(ValueError):
        q.qlora_fp8_gated_fwd(w, w, x, act="relu")
    with pytest.raises(ValueError):
        q.qlora_fp8_gated_fwd(w, _fp8(144, 64), x)


def _nf4(rows, cols, **kw):
    return q.NF4Weight.empty(rows, cols, device="cpu", **kw)


def test_gated_binding_refusals():
    bf = torch.bfloat16
    w = [_nf4(128, 64), _nf4(128, 64)]
    x, a, b = torch.zeros(4, 64, dtype=bf), torch.zeros(16, 64, dtype=bf), torch.zeros(128, 16, dtype=bf)
    h = torch.zeros(4, 128, dtype=bf)
    u = torch.zeros(4, 16, dtype=bf)
    saved = q.GatedSaved(h, h, u, u)

    def fwd(w=w, x=x, a=a, b=b, **kw):
        return q.qlora_gated_linear_fwd(*w, x, a, b, a, b, 16.0, **kw)

    def bwd(saved=saved, dh=h, **kw):
        return q.qlora_gated_linear_bwd(*w, x, dh, a, b, a, b, 16.0, saved, **kw)

    for call, error in ((lambda: fwd(act="tanh"), ValueError),
                        (lambda: fwd(w=[w[0], _nf4(144, 64)]), ValueError),
                        (lambda: fwd(x=x.half()), TypeError),
                        (lambda: fwd(a=a[:, :32].contiguous()), ValueError),
                        (lambda: fwd(a=a.T), ValueError), (lambda: fwd(a=a[None]), ValueError),
                        (lambda: fwd(b=b.float()), TypeError),
                        (lambda: fwd(H=x), ValueError),
                        (lambda: fwd(saved=q.GatedSaved(h, h, u, h)), ValueError),
                        (lambda: fwd(), ValueError),                # not on a GPU
                        (lambda: bwd(act="relu"), ValueError),
                        (lambda: bwd(dh=x), ValueError),
                        (lambda: bwd(saved=q.GatedSaved(h, h.float(), u, u)), TypeError),
                        (lambda: bwd(dX=h), ValueError),
                        (lambda: bwd(dA_up=a), TypeError),
                        (lambda: bwd(), ValueError)):
        with pytest.raises(error):
            call()


# --------------------------------------------------------------------------
# the references
# --------------------------------------------------------------------------
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_gated_reference_against_differences(name):
    """The backward's formulas against central differences of <dH, H>, and the
    activation against torch's."""
    g = torch.Generator().manual_seed(3)
    f64 = torch.float64
    T, N, K, r, scale = 5, 6, 7, 3, 0.7

    def rand(*shape):
        return torch.randn(shape, generator=g, dtype=f64)

    x, w = rand(T, K), [rand(N, K), rand(N, K)]
    A, B, dh = [rand(r, K), rand(r, K)], [rand(N, r), rand(N, r)], rand(T, N)
    z = rand(1000) * 5
    ref = torch.nn.functional.silu(z) if name == "silu" else \
        torch.nn.functional.gelu(z, approximate="tanh")
    assert torch.allclose(G.act(z, name)[0], ref, atol=1e-14)

    def loss():
        return (dh * G.forward(x, w, A, B, scale, name, torch.bfloat16)[0][0]).sum().item()

    (_, P, U), _ = G.forward(x, w, A, B, scale, name, torch.bfloat16)
    (dX, dA, dB), _ = G.backward(x, dh, w, A, B, scale, name, P, U, torch.bfloat16)
    step = 1e-6
    for t, grad in ((x, dX), (A[0], dA[0]), (A[1], dA[1]), (B[0], dB[0]), (B[1], dB[1])):
        flat = t.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + step
            up = loss()
            flat[i] = keep - step
            down = loss()
            flat[i] = keep
            assert abs((up - down) / (2 * step) - grad.reshape(-1)[i].item()) < 1e-6


def test_e4m3_values_and_rounding():
    """The enumerated values are torch's, and the nearest one is its conversion."""
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(bits.double().numpy(), R.E4M3)
    x = np.concatenate([(R.E4M3[1:] + R.E4M3[:-1]) / 2, R.E4M3,
                        np.random.default_rng(0).standard_normal(4000) * 30])
    x = np.concatenate([x, -x]).astype(np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(1e9)), np.nextafter(x, np.float32(-1e9))])
    x = np.clip(x, -448, 448)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3_nearest(x.astype(np.float64)), ref)


def test_quantize_reference_on_a_hand_case():
    x = np.zeros((2, 144), np.float32)
    x[0, :4] = [896, -3, 1, 0.001]       # scale 2
    x[1, 130] = -7                       # scale 1/64
    c, s = R.quantize(x, 1)
    assert s.tolist() == [[2.0, 0.0], [0.0, 1 / 64]]
    assert c[0, :4].tolist() == [448, -1.5, 0.5, 0] and c[1, 130] == -448
    c, s = R.quantize(x, 128)
    assert s.tolist() == [[2.0, 1 / 64]] and c[1, 130] == -448

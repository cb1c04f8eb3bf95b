"""The linear layer and the gated block in 8-bit floating point in 64 bits:
codes by enumeration of the E4M3 values, products and their error bounds."""
import math

import numpy as np
import torch

TILE = 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
# the finite E4M3 values of sign 0, by bit pattern 0 .. 126
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def e4m3_nearest(q):
    """E4M3 values nearest to q (float64, |q| <= 448), ties to the even pattern."""
    a = np.abs(q)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    take = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.sign(q) * E4M3[take]


def blocks(x, br):
    rows, cols = x.shape
    p = np.zeros((-(-rows // br) * br, -(-cols // TILE) * TILE))
    p[:rows, :cols] = x
    return p.reshape(p.shape[0] // br, br, p.shape[1] // TILE, TILE)


def quantize(x, br):
    """x float32 [rows, cols] -> (code values [rows, cols], scale float32
    [row blocks, column blocks]); br rows share a scale."""
    b = blocks(x.astype(np.float64), br)
    with np.errstate(over="ignore", under="ignore"):
        scale = (np.abs(b).max((1, 3)) / 448).astype(np.float32)
        s = scale.astype(np.float64)[:, None, :, None]
        q = np.where(s > 0, b / np.where(s > 0, s, 1), 0).astype(np.float32).astype(np.float64)
    c = e4m3_nearest(np.clip(q, -448, 448)).reshape(b.shape[0] * br, -1)
    return c[:x.shape[0], :x.shape[1]], scale


def every(scale, br, shape):
    """scale [row blocks, column blocks] for each element"""
    s = scale.double().repeat_interleave(br, 0)[:shape[0]]
    return s.repeat_interleave(TILE, 1)[:, :shape[1]]


def values(codes, scale, br):
    """codes (float8 tensor) and scale [row blocks, column blocks] -> float64
    values, and for each 8 consecutive columns the largest power of two not
    above a code (2^-6 at least: the exponent that a subnormal code has), scaled."""
    v, s = codes.float().double(), every(scale, br, codes.shape)
    power = torch.exp2(torch.frexp(v).exponent.double() - 1).clamp_min(2.0 ** -6)
    group = (power * s).view(len(v), -1, 8).amax(2)
    return v * s, group


def product(x, w):
    """P = x w^T of values() and the bound of its evaluation.

    The sums of 128 products, the product of the scales (one rounding) and the
    sums over the blocks and parts are float32: at most 2^-23 of the sum of the
    magnitudes each.  But the matrix core adds 8 products of consecutive codes
    as fixed-point numbers first, all cut towards zero at 2^-13 of 2^E, E the
    largest sum of two codes' exponents among the 8 (measured with one product
    of 2^16 and another of +-2^3, kept, or +-2^2, lost, at every distance below
    8, and kept down to float32's last place at 8 and more; the products of 8
    bits with E = 16 themselves are exact).  So of each 8 products 7 lose less
    than 2^-13 2^E, and 2^E is at most the product of the two groups' largest
    powers of two."""
    (x, gx), (w, gw) = x, w
    terms = 128 + -(-x.shape[1] // TILE) + 20
    err = 7 * 2.0 ** -13 * (gx @ gw.T) + terms * 2.0 ** -23 * (x.abs() @ w.abs().T)
    return x @ w.T, err


def act(g, name):
    z = g if name == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(z), z


def gated(x, wg, wu, name):
    """H and its bound before the final rounding.  |act'| < 1.2 (its largest
    value is 1.13 for GELU, 1.10 for SiLU); the float32 sigmoid is off by a few
    2^-23 and by the rounding of its argument, |z| 2^-23 times a few."""
    (g, eg), (u, eu) = product(x, wg), product(x, wu)
    a, z = act(g, name)
    ea = 1.2 * eg + a.abs() * (6 + 6 * z.abs().clamp_max(90)) * 2.0 ** -23
    return a * u, ea * (u.abs() + eu) + a.abs() * eu


def check(y, ref, err, what):
    """y is ref within err, plus half a step of its own type (fp16 below its
    normal range: 2^-25)."""
    lim = err + HALF[y.dtype] * (ref.abs() + err) + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    bad = ~((y.double() - ref).abs() <= lim)
    worst = ((y.double() - ref).abs() / lim.clamp_min(1e-300)).max().item() if y.numel() else 0
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), worst)

"""The gated feed-forward block in 64 bits, and how far its evaluation in float32
with 16-bit operands may be off, element by element."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}         # half the smallest step
# a value as two 16-bit terms: half a step of the rest of half a step; fp16's
# second term is taken times 2^11, so its smallest half step is 2^-36
TWO = {torch.bfloat16: (2.0 ** -16, 0.0), torch.float16: (2.0 ** -22, 2.0 ** -36)}
U32 = 2.0 ** -23                                                # a float32 sum, per term


def act(g, name):
    """act(g), its slope, and z and its slope: act = g sigmoid(z)."""
    z, dz = g, torch.ones_like(g)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(z)
    return g * s, s + g * s * (1 - s) * dz, z, dz


def act_error(g, name):
    """Float32 evaluation: the sigmoid's argument is off by a few roundings of
    z (its own, the product with log2 e, the cube), |z| of 2^-23 a few times,
    which the sigmoid's slope s (1 - s) |z| <= s |z| passes on; exponential,
    sum, reciprocal and product add a few 2^-23.  1 - s is off by 2^-24
    absolutely."""
    a, slope, z, dz = act(g, name)
    rel = (8 + 6 * z.abs().clamp_max(90)) * U32
    s = torch.sigmoid(z)
    return a.abs() * rel, rel * (s + (g * s * (1 - s) * dz).abs()) + (g * s * dz).abs() * U32


def mm(a, b):
    return a @ b


def forward(x, w, A, B, scale, name, dt):
    """x, w[2], A[2], B[2] as float64 values of 16-bit tensors.  Returns
    (H, P, U) and their bounds before the last rounding."""
    K, r = x.shape[1], A[0].shape[0]
    P, U, eP, eU = [], [], [], []
    for i in range(2):
        u = mm(x, A[i].T)
        du = K * U32 * mm(x.abs(), A[i].abs().T)
        su, dsu = scale * u, abs(scale) * du
        dsu = dsu + HALF[dt] * (su.abs() + dsu) + TINY[dt]
        P.append(mm(x, w[i].T) + mm(su, B[i].T))
        eP.append(K * U32 * mm(x.abs(), w[i].abs().T) + mm(dsu, B[i].abs().T)
                  + r * U32 * mm(su.abs(), B[i].abs().T) + 4 * U32 * P[i].abs())
        U.append(u)
        eU.append(du)
    a = act(P[0], name)[0]
    ea = 1.2 * eP[0] + act_error(P[0], name)[0]     # |act'| < 1.2
    eH = ea * (P[1].abs() + eP[1]) + a.abs() * eP[1]
    return (a * P[1], P, U), (eH, eP, eU)


def backward(x, dh, w, A, B, scale, name, P, U, dt):
    """Returns (dX, dA[2], dB[2]) and their bounds before the last rounding."""
    T, N, r = x.shape[0], dh.shape[1], A[0].shape[0]
    a, slope, _, _ = act(P[0], name)
    ea, es = act_error(P[0], name)
    d = [dh * P[1] * slope, dh * a]
    ed = [(dh * P[1]).abs() * es + 2 * U32 * d[0].abs(), dh.abs() * ea + 2 * U32 * d[1].abs()]
    two, two0 = TWO[dt]
    dx, ex = torch.zeros_like(x), torch.zeros_like(x)
    dA, dB, eA, eB = [], [], [], []
    for i in range(2):
        one = ed[i] + HALF[dt] * d[i].abs() + TINY[dt]           # as one 16-bit value
        pair = ed[i] + two * d[i].abs() + two0                   # as two terms
        g = mm(d[i], B[i])
        eg = mm(pair, B[i].abs()) + N * U32 * mm(d[i].abs(), B[i].abs())
        sg, esg = scale * g, abs(scale) * eg
        dx += mm(d[i], w[i]) + mm(sg, A[i])
        ex += mm(one, w[i].abs()) + 2 * N * U32 * mm(d[i].abs(), w[i].abs())
        ex += mm(esg + HALF[dt] * (sg.abs() + esg) + TINY[dt], A[i].abs())
        ex += r * U32 * mm(sg.abs(), A[i].abs())
        dA.append(scale * mm(g.T, x))
        eA.append(abs(scale) * (mm((eg + two * g.abs() + two0).T, x.abs())
                                + T * U32 * mm(g.abs().T, x.abs())) + 4 * U32 * dA[i].abs())
        dB.append(scale * mm(d[i].T, U[i]))
        eB.append(abs(scale) * (mm(pair.T, U[i].abs()) + T * U32 * mm(d[i].abs().T, U[i].abs()))
                  + 4 * U32 * dB[i].abs())
    return (dx, dA, dB), (ex, eA, eB)


def check(y, ref, err, what):
    half, tiny = HALF.get(y.dtype, 2.0 ** -24), TINY.get(y.dtype, 0.0)
    lim = err + half * (ref.abs() + err) + tiny
    off = (y.double() - ref).abs()
    bad = ~(off <= lim)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           (off / lim.clamp_min(1e-300)).max().item())


def near(y, ref, tol, what):
    """over the whole tensor, in norm"""
    rel = ((y.double() - ref).norm() / ref.norm()).item()
    assert rel <= tol, (what, rel)

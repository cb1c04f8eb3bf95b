"""Cases of the gated block over NF4 weights in which only what the adapters'
products keep of U = X A^T and G = d B can be off: the weights are zero, U and G
are whole numbers times a power of two, exact in float32 and of more bits than
16-bit types hold, the gate is 64 (an activation of exactly 64, a slope of exactly
1), and each output is the sum of two of U's (G's) columns."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}         # half the smallest step
U32 = 2.0 ** -23                                                # a float32 sum, per term


def integers(gen, shape, red, dev):
    """Whole numbers whose products' sums over `red` stay below 2^24."""
    top = min(127, int((2 ** 24 / red) ** 0.5))
    return torch.randint(-top, top + 1, shape, generator=gen, device=dev).double()


def pairs(gen, n, r, dev):
    """[n, r] of two entries +-1 a row (one where r = 1); the rows meet every
    column."""
    out = torch.zeros(n, r, dtype=torch.float64, device=dev)
    rows = torch.arange(n, device=dev)
    sign = torch.randint(0, 2, (2, n), generator=gen, device=dev).double() * 2 - 1
    first = rows % r
    out[rows, first] = sign[0]
    if r > 1:
        out[rows, (first + 1 + rows // r % (r - 1)) % r] = sign[1]
    return out


def forward_case(T, N, K, r, seed, dev, x=1.0, a=1.0, b=1.0):
    """X, A[2], B[2] in float64."""
    g = torch.Generator(device=dev).manual_seed(seed + T + N + K + r)
    X = integers(g, (T, K), K, dev) * x
    A = [integers(g, (r, K), K, dev) * a for _ in range(2)]
    return X, A, [pairs(g, N, r, dev) * b for _ in range(2)]


def backward_case(T, N, K, r, seed, dev, d=1.0, a=1.0, b=1.0, up=64.0):
    """dH, A[2], B[2], P[2]: dG = up dH and dU = 64 dH exactly."""
    g = torch.Generator(device=dev).manual_seed(seed + T + N + K + r)
    dH = integers(g, (T, N), N, dev) * d
    B = [integers(g, (N, r), N, dev) * b for _ in range(2)]
    A = [pairs(g, K, r, dev).T.contiguous() * a for _ in range(2)]
    return dH, A, B, [torch.full((T, N), v, dtype=torch.float64, device=dev) for v in (64.0, up)]


def off(v, mag, dt):
    """How far two 16-bit terms of v may be from it: half a step of half a step.  In
    fp16 they are those of v times a power of two for 128 rows that brings S times
    the rows' largest of S partial sums below 2^15, and a term is no closer than
    2^-25, which is 2^-39 of that product's next power of two: 2^-38 S of the
    partials, S <= 64 of them, each at most the largest sum of magnitudes, mag."""
    e = HALF[dt] ** 2 * v.abs()
    if dt == torch.float16:
        e = e + torch.cat([torch.full_like(m, float(m.max())) for m in mag.split(128)]) * 2.0 ** -32
    return e


def projections(X, A, B, scale, dt):
    """P = s U B^T of either adapter and its bound before the last rounding: two
    terms of two columns, and the products with s and the power of two, in float32."""
    out = []
    for a, b in zip(A, B):
        u, mag = X @ a.T, X.abs() @ a.abs().T
        err = abs(scale) * ((off(u, mag, dt) + 8 * U32 * u.abs()) @ b.abs().T)
        out.append((scale * (u @ b.T), err))
    return out


def dx(dH, A, B, P, scale, dt):
    """dX = s sum_i (d_i B_i) A_i and its bound; in fp16 the rows of both share
    their power of two."""
    grads = [dH * P[1], dH * P[0]]
    mag = torch.maximum(*(d.abs() @ b.abs() for d, b in zip(grads, B)))
    val, err = 0, 0
    for d, a, b in zip(grads, A, B):
        G = d @ b
        val = val + scale * (G @ a)
        err = err + abs(scale) * ((off(G, mag, dt) + 12 * U32 * G.abs()) @ a.abs())
    return val, err


def da(dH, X, B, P, scale, dt):
    """dA = s (d B)^T X of either adapter, X two tokens a column, and its bound: three
    terms of G in bf16 (2^-24), two in fp16, their products and the tiles' and parts'
    sums in float32."""
    grads = [dH * P[1], dH * P[0]]
    mag = torch.maximum(*(d.abs() @ b.abs() for d, b in zip(grads, B)))
    out = []
    for d, b in zip(grads, B):
        G = d @ b
        e = 2.0 ** -24 * G.abs() if dt == torch.bfloat16 else off(G, mag, dt)
        out.append((scale * (G.T @ X), abs(scale) * ((e + 12 * U32 * G.abs()).T @ X.abs())))
    return out


def picked_case(T, N, K, r, seed, dev, dt):
    """Gradients that are single values of d = dG, dU, which need float32's 24 bits: U
    is the unit matrix over the first r tokens, B over the first r rows, X over the
    first K tokens (T, N, K >= r), so dB_np = s d_pn and dA_pk = s d_kp."""
    g = torch.Generator(device=dev).manual_seed(seed + T + N + K + r)

    def rand(lo):
        return (lo + (1 - lo) * torch.rand(T, N, generator=g, device=dev)).to(dt).double()

    dH, P = rand(0.5), [rand(0.125), rand(0.5)]
    eye = lambda n, m: torch.eye(n, m, dtype=torch.float64, device=dev)  # noqa: E731
    s = torch.sigmoid(P[0])
    d = [dH * P[1] * (s + P[0] * s * (1 - s)), dH * P[0] * s]
    return dH, P, eye(T, r), eye(N, r), eye(T, K), d


def picked(d, r, K, dt):
    """(dA, dB) / s of either adapter, and their bounds relative to the value, in units
    of 2^-24.  SiLU with z = P_gate in 0 .. 1: the exponent, z log2 e, is off by its
    rounding and the constant's, |z| 1.4; exponential and reciprocal by one unit in
    the last place each, 2; the sum by 1; so the sigmoid s by (1 - s) 3.4 + 3 <= 4.7.
    dU takes two products, 6.7.  The slope s + (g s)(1 - s): with 1 - s off by 4.7 s /
    (1 - s) + 1, at most 8 of the sum, 9 after its rounding, 10 after the product with
    dH P_up, which is exact.  That is 11 at most; bf16's terms add nothing (24
    bits), fp16's two 4 in dB, and 4 more in dA, where d B is split again."""
    f16 = dt == torch.float16
    n = min(r, d[0].shape[0])
    k = min(K, d[0].shape[0])
    out = []
    for v in d:
        dB = torch.zeros(v.shape[1], r, dtype=torch.float64, device=v.device)
        dB[:, :n] = v[:n].T
        dA = torch.zeros(r, K, dtype=torch.float64, device=v.device)
        dA[:, :k] = v[:k, :r].T
        out.append(((dA, (11 + 8 * f16) * 2.0 ** -24 * dA), (dB, (11 + 4 * f16) * 2.0 ** -24 * dB)))
    return out


def check(y, ref, err, what):
    half, tiny = HALF.get(y.dtype, 2.0 ** -24), TINY.get(y.dtype, 0.0)
    lim = err + half * (ref.abs() + err) + tiny
    diff = (y.double() - ref).abs()
    bad = ~(diff <= lim)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           (diff / lim.clamp_min(1e-300)).max().item())

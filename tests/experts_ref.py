"""Plain 64-bit forms of the expert-grouped linear layer, and the bounds its
kernels are held to."""
import numpy as np


def groups(off):
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1)]


def grouped_forward(X, W, A, B, off, alpha):
    """Y, U of rows off[e] .. off[e + 1] - 1 with W[e] [N, K], A[e] [r, K],
    B[e] [N, r]; rows that no expert owns are 0."""
    Y = np.zeros((X.shape[0], W.shape[1]))
    U = np.zeros((X.shape[0], A.shape[1]))
    for e, i, j in groups(off):
        U[i:j] = X[i:j] @ A[e].T
        Y[i:j] = X[i:j] @ W[e].T + alpha / A.shape[1] * (U[i:j] @ B[e].T)
    return Y, U


def grouped_backward(X, dY, W, A, B, off, alpha, U):
    """dX, dA, dB for the forward's U."""
    s = alpha / A.shape[1]
    dX, dA, dB = np.zeros(X.shape), np.zeros(A.shape), np.zeros(B.shape)
    for e, i, j in groups(off):
        G = dY[i:j] @ B[e]
        dX[i:j] = dY[i:j] @ W[e] + s * G @ A[e]
        dA[e] = s * G.T @ X[i:j]
        dB[e] = s * dY[i:j].T @ U[i:j]
    return dX, dA, dB


# A float32 sum of n terms is off by at most about n u sum |terms|, u = 2^-24;
# twice that also covers a matrix core that truncates.
U_ACC = 2.0 ** -23


def group_bounds(x, dy, w, a, b, alpha, half):
    """Absolute bounds per element of one expert's Y, U, dX, dA, dB against
    the 64-bit formulas.  half: half a step of the 16-bit type relative to the
    value (2^-8 for bf16, 2^-11 for fp16).  sum |p q| <= |p| |q| (Cauchy-
    Schwarz) turns every accumulation into an outer product of norms.

    U: the sum over K, one rounding.  Y: the sum over K + r with s U rounded
    twice on its way (U to 16 bits is not what meets B: s U is, one rounding of
    the float32 sum), and the output's rounding.  dX likewise with s G.
    dA: G keeps at least 22 bits (2^-22), its own sum over N, the sum over the
    rows (each with up to 3 terms).  dB: U is given, only the sum over rows."""
    r, (T, K), N = a.shape[0], x.shape, w.shape[0]
    s = abs(alpha) / r
    n = lambda m, ax: np.sqrt((m * m).sum(ax))  # noqa: E731
    nx, ndy = n(x, 1), n(dy, 1)
    u, g = x @ a.T, dy @ b
    acc_u = K * U_ACC * np.outer(nx, n(a, 1))
    acc_g = N * U_ACC * np.outer(ndy, n(b, 0))
    y = x @ w.T + alpha / r * (u @ b.T)
    dx = dy @ w + alpha / r * (g @ a)
    out = {"u": acc_u + half * np.abs(u)}
    eu = s * (half * np.abs(u) + 1.01 * acc_u)
    eg = s * (half * np.abs(g) + 1.01 * acc_g)
    out["y"] = (1.01 * (K + r) * U_ACC * (np.outer(nx, n(w, 1)) + s * np.outer(n(u, 1), n(b, 1)))
                + eu @ np.abs(b).T + half * np.abs(y))
    out["dx"] = (1.01 * (N + r) * U_ACC * (np.outer(ndy, n(w, 0)) + s * np.outer(n(g, 1), n(a, 0)))
                 + eg @ np.abs(a) + half * np.abs(dx))
    if T:
        out["da"] = s * 1.01 * ((2.0 ** -22 + (3 * T + 16) * U_ACC) * np.outer(n(g, 0), n(x, 0))
                                + acc_g.T @ np.abs(x))
    else:
        out["da"] = np.zeros(a.shape)
    return out


def db_bound(dy, u, alpha, r):
    s = abs(alpha) / r
    n = lambda m: np.sqrt((m * m).sum(0))  # noqa: E731
    return s * 1.01 * (dy.shape[0] + 16) * U_ACC * np.outer(n(dy), n(u))

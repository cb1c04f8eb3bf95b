"""The fast conversion of the row quantiser next to the borders between codes.

A code is taken from one FMA, x * inv + 1.5 * 2^23, where the remainder
x * inv - r is at most 0.49996 in size; otherwise the exact rule decides.  inv
is the rounded reciprocal of the scale (2^-24 relative, and half an ulp of the
quotient), so x * inv is within 127 * 2^-23 < 2^-16 of the quotient and the
remainder is rounded once more: below 0.5 - 2^-16 - 2^-25 > 0.49998 the nearest integer is r."""
import numpy as np

from test_kernel_arith_host import fma32

F = np.float32
MAGIC, CLEAR = F(12582912.0), F(0.49996)


def border_rows(seed, n):
    """(x, scale) at (k + 1/2 + delta) * scale for deltas from 0 past the fast
    path's limit, rounded to float32, and the floats beside."""
    rng = np.random.default_rng(seed)
    s = np.concatenate([(1 + rng.random(n)).astype(F),
                        np.exp2(rng.integers(-99, 100, n)).astype(F) * (1 + rng.random(n)).astype(F)])
    k = rng.integers(-127, 127, s.size)
    xs, ss = [], []
    for delta in (0, 1e-7, 1e-6, 1e-5, 1.9e-5, 3.9e-5, 3.99e-5, 4e-5, 4.01e-5, 4.1e-5, 1e-4, 1e-2):
        for sign in (-1, 1):
            x = ((k + 0.5 + sign * delta) * s.astype(np.float64)).astype(F)
            for y in (x, np.nextafter(x, F(np.inf)), np.nextafter(x, F(-np.inf))):
                xs.append(y)
                ss.append(s)
    x, s = np.concatenate(xs), np.concatenate(ss)
    keep = np.abs(x.astype(np.float64)) <= 127 * s.astype(np.float64)
    return x[keep], s[keep]


def test_fast_codes_are_exact_up_to_their_limit():
    x, s = border_rows(11, 1500)
    inv = (F(1) / s).astype(F)
    m = fma32(x, inv, np.full_like(x, MAGIC))
    d = fma32(x, inv, -(m - MAGIC).astype(F))
    fast = np.abs(d) <= CLEAR
    code = (m.view(np.uint32) & 255).astype(np.uint8).view(np.int8).astype(np.int64)
    # x and s hold 24 bits: numerators and denominators are small enough for
    # Python's integers to settle every case
    tested = 0
    for i in np.flatnonzero(fast):
        xn, xd = float(x[i]).as_integer_ratio()
        sn, sd = float(s[i]).as_integer_ratio()
        num, den = xn * sd, xd * sn
        low = num // den
        twice = 2 * (num - low * den)
        want = low + (1 if twice > den or (twice == den and low % 2) else 0)
        assert code[i] == want, (x[i], s[i], code[i], want, d[i])
        # how many lie close to the limit on the inside
        tested += abs(abs(float(d[i])) - 0.49996) < 3e-6
    assert tested > 100 and (~fast).sum() > 1000, (tested, int((~fast).sum()))

"""Plain 64-bit forms of the experts' layer in 8-bit integers, for the tests to compare
with.  numpy only; nothing here is shared with the library.

Bounds.  u = 2^-24 is half a step of fp32, relative to the value.  A product's sum is an
exact integer; on its way to fp32, in the product of the two scales and in theirs it is
rounded three times: 3 u of the value.
silu(g) * up, g off by 3 u: 3 u (1 + |g|) of silu; the exponent -1.44 g by two roundings,
2 u |g| of the exponential; the hardware's exponential and reciprocal a step of 2 u
each, an addition, two products: 7 u; up 3 u.  (13 + 5 |g|) u in all; 16 + 6 |g| is used.
Below g = -88 the exponential leaves fp32, and silu, at most 88 e^-88 < 2^-120, is 0."""
import numpy as np

U = 2.0 ** -24


def bf16(a):
    """The bf16 nearest to fp64 `a` (through fp32, whose roundings are the caller's)."""
    b = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32).astype(np.float64)


def cast(x):
    """x [rows, K] fp64 (values of bf16) -> codes int64 and scales fp32."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.shape, np.int64)
    a = np.abs(x).max(axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        scales = a.astype(np.float32) / np.float32(127)
        for r in range(len(x)):
            if a[r] > 0 and np.isfinite(a[r]):
                codes[r] = np.rint(127.0 * x[r] / a[r])     # halves come out exactly, to even
    return codes, scales


def linear(x, xs, spans, w, ws, silu):
    """x [rows, K] int, xs [rows], spans [(first, count)], w [E, W, K] int, ws [E, W]:
    (v [rows, N] fp64 with NaN where no expert has the row, bound on its error before
    the rounding to bf16)."""
    W = w.shape[1]
    N = W // 2 if silu else W
    y, tol = np.full((len(x), N), np.nan), np.zeros((len(x), N))
    for (first, count), we, se in zip(spans, w, ws):
        if not count:
            continue
        rows = slice(first, first + count)
        v = (x[rows].astype(np.float64) @ we.astype(np.float64).T) * (xs[rows].astype(np.float64)[:, None] * se.astype(np.float64))
        if silu:
            g, up = v[:, :N], v[:, N:]
            with np.errstate(over="ignore"):
                s = g / (1.0 + np.exp(-g))
            y[rows] = s * up
            tol[rows] = (16 + 6 * np.abs(g)) * U * np.abs(s * up) + 2.0 ** -118 * np.abs(up)
        else:
            y[rows], tol[rows] = v, 3.01 * U * np.abs(v)
    return y, tol


def moe(x, idx, weights, up, us, down, ds):
    """The whole layer: (out [T, H] fp64, bound on the error before the rounding to bf16)."""
    T, k = idx.shape
    E, W, H = up.shape
    F = W // 2
    xq, xs = cast(x)
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            wt = 1.0 if weights is None else float(weights[t, j])
            h, dh = linear(xq[t:t + 1], xs[t:t + 1], [(0, 1)], up[e:e + 1], us[e:e + 1], True)
            h, dh = h[0], dh[0]
            a = np.abs(h).max()
            if not np.isfinite(a):
                out[t] = np.nan
                continue
            da = dh[np.abs(h) + dh >= a - dh.max()].max()           # whichever is the largest in fp32
            if a == 0:
                continue
            q = 127.0 * h / a
            code = np.rint(q)
            # A code may come out one off where the quotient's error reaches a half.
            slack = 127.0 * (dh / a + np.abs(h) * da / a ** 2) + 4 * U * 127
            near = np.abs(np.abs(q - code) - 0.5) <= slack
            scale = a / 127.0 * ds[e].astype(np.float64)
            d = down[e].astype(np.float64)
            y = (d @ code) * scale
            dy = (np.abs(d) @ near.astype(np.float64)) * scale * 1.001 + (da / a + 5 * U) * np.abs(y)
            out[t] += wt * y
            tol[t] += abs(wt) * (dy + (k + 1) * U * np.abs(y))
    return out, tol

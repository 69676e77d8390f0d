"""64-bit NumPy forms of the gated linear recurrence and of the norms around a
mixer block, each with a bound on what fp32 arithmetic may be off.

u = 2^-24 is half an fp32 step.  Bounds follow the errors through the formulas
(first order in u) with C roundings charged wherever a value is formed; the
last rounding to the output's type adds half a step of that type."""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def check(got, want, err, io, what=""):
    """Every element of ``got`` within its bound; where ``want`` is not finite, the same."""
    got, want = np.asarray(got, np.float64).reshape(want.shape), np.asarray(want)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), what
    off = np.abs(got - want)[fine]
    most = rounded(want, np.broadcast_to(err, want.shape), io)[fine] + 1e-38  # subnormal results
    bad = ~(off <= most)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(off / most):.3g} of the bound"


def rounded(value, err, io):
    """Bound of a value of magnitude |value| known to err, rounded to ``io``."""
    return err + HALF_STEP[io] * (np.abs(value) + err)


# A decay exp(g) is within 2 ulp (4 u); that of a span of tokens is exp of a sum
# of at most 64 terms, off by at most 64 u |sum|, and x exp(-x) < 0.37: 24 u.  A
# state takes one product-sum a token and at most four more of a span: 12 u a
# token cover a span of one token; a span of more shares its 24 u.
C_SCAN = 40


def scan(x, g, h0, cu, complement):
    """x, g [M, D]; h0 [N, D]; cu [N + 1].  Returns (h, final, bound of h, bound of final)."""
    x, g, h0 = (np.asarray(a, np.float64) for a in (x, g, h0))
    h, e = np.empty_like(x), np.empty_like(x)
    final, efinal = h0.copy(), np.zeros_like(h0)
    a = np.exp(g)
    b = -np.expm1(g) * x if complement else x
    for n in range(len(cu) - 1):
        s, m, err = h0[n], np.abs(h0[n]), np.zeros(x.shape[1])
        for t in range(cu[n], cu[n + 1]):
            s = a[t] * s + b[t]
            m = a[t] * m + np.abs(b[t])
            err = a[t] * err + C_SCAN * U * m
            h[t], e[t] = s, err
        final[n], efinal[n] = s, err
    return h, final, e, efinal


def scan_bwd(dh, dfinal, x, g, h0, cu, complement):
    """Returns ((dx, dg, dh0), (their bounds))."""
    dh, dfinal, x, g, h0 = (np.asarray(a, np.float64) for a in (dh, dfinal, x, g, h0))
    h, _, eh, _ = scan(x, g, h0, cu, complement)
    a, u = np.exp(g), -np.expm1(g) if complement else np.ones_like(g)
    dx, dg, ex, eg = (np.empty_like(x) for _ in range(4))
    dh0, e0 = dfinal.copy(), np.zeros_like(dfinal)
    for n in range(len(cu) - 1):
        c, m, err = dfinal[n], np.abs(dfinal[n]), np.zeros(x.shape[1])
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            d, m = dh[t] + c, np.abs(dh[t]) + m
            err = err + C_SCAN * U * m
            dx[t], ex[t] = u[t] * d, u[t] * (err + 8 * U * m)
            before = h[t - 1] if t > cu[n] else h0[n]
            ebefore = eh[t - 1] if t > cu[n] else 0.0
            f = before - x[t] if complement else before
            size = np.abs(before) + np.abs(x[t]) if complement else np.abs(before)
            dg[t] = d * a[t] * f
            eg[t] = a[t] * (err * size + m * ebefore + 12 * U * m * size)
            c, m, err = a[t] * d, a[t] * m, a[t] * (err + 8 * U * m)
        dh0[n], e0[n] = c, err
    return (dx, dg, dh0), (ex, eg, e0)


# A mean of squares is a sum of positive terms: a thread adds at most 32, ten
# more additions join the threads; with the division, the root and the products
# a normalised value is off by less than 64 u of itself.
C_NORM = 64
# sigmoid: the accurate functions are within 4 ulp; the intrinsics of the bf16
# path within 2^-20 (1 + |z|), far below a bf16 rounding.


def _c_gate(z, io):
    return np.full_like(z, 16 * U) if io == "f32" else 2.0 ** -20 * (1 + np.abs(z))


def _gate(z, kind):
    if kind is None:
        return np.ones_like(z), np.zeros_like(z)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def gated_norm(x, z, w, kind, eps, io):
    x, z, w = (np.asarray(a, np.float64) for a in (x, z, w))
    s, _ = _gate(z, kind)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w * s
    return y, np.abs(y) * (C_NORM * U + _c_gate(z, io))


def gated_norm_bwd(dy, x, z, w, kind, eps, io, chain):
    """[rows, d] arrays; ``chain``: additions that a column sum may take one after another."""
    dy, x, z, w = (np.asarray(a, np.float64) for a in (dy, x, z, w))
    inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, (s, ds) = x * inv, _gate(z, kind)
    du = dy * w * s
    k = C_NORM * U + _c_gate(z, io)
    k_row = k.max(-1, keepdims=True)
    dx = inv * (du - u * (du * u).mean(-1, keepdims=True))
    ex = inv * (np.abs(du) * k + np.abs(u) * np.abs(du * u).mean(-1, keepdims=True) * 3 * k_row)
    dz = dy * u * w * ds
    # the slope is a difference: its terms' sizes count, not its own
    slope = (1 + np.abs(z)) if kind == "silu" else np.ones_like(z)
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-z))
    ez = np.abs(dy * u * w) * sig * slope * 3 * k if kind else np.zeros_like(x)
    dw = (dy * u * s).sum(0)
    ew = (np.abs(dy * u * s) * (k + chain * U)).sum(0)
    return (dx, dz, dw), (ex, ez, ew)


def add_norm(r, y, w, scale, eps):
    r, y, w, scale = (np.asarray(a, np.float64) for a in (r, y, w, scale))
    t = r + scale * y
    et = 2 * U * (np.abs(r) + np.abs(scale * y))
    inv = 1 / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    n = t * inv * w
    en = (et + np.abs(t) * (C_NORM * U + (np.abs(t) * et).mean(-1, keepdims=True) * inv ** 2)) * inv * np.abs(w)
    return (t, n), (et, en)


def add_norm_bwd(dn, dt, t, y, w, scale, chain, eps):
    dn, dt, t, y, w, scale = (np.asarray(a, np.float64) for a in (dn, dt, t, y, w, scale))
    inv = 1 / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    u, du, k = t * inv, dn * w, C_NORM * U
    d = dt + inv * (du - u * (du * u).mean(-1, keepdims=True))
    ed = k * (np.abs(dt) + inv * (np.abs(du) + 3 * np.abs(u) * np.abs(du * u).mean(-1, keepdims=True)))
    dy, ey = scale * d, np.abs(scale) * ed + 2 * U * np.abs(scale * d)
    dw, ew = (dn * u).sum(0), (np.abs(dn * u) * (k + chain * U)).sum(0)
    ds, es = (d * y).sum(0), (np.abs(y) * ed + np.abs(d * y) * chain * U).sum(0)
    return (d, dy, dw, ds), (ed, ey, ew, es)

"""Float64 references of the operators around the router and the experts: the residual RMS norm,
the products with 4-bit weights and the balance loss (test infrastructure; numpy only)."""
import numpy as np


def rms_norm(x, residual, weight, eps):
    s = x if residual is None else x + residual
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s, y if weight is None else y * weight


def groups(d, group):
    """Column ranges of the 8-bit scales."""
    g = group or d
    return [(i, min(i + g, d)) for i in range(0, d, g)]


def e4m3_to_f64(b):
    """Values of e4m3 bytes, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = b.astype(np.int64)
    s, e, m = np.where(b >> 7, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where((b & 127) == 127, np.nan, s * v)


def w4_values(q, scale, rows, cols, group):
    """[mats, parts, rows, cols] values of stored 4-bit matrices, byte by byte."""
    mats, parts, rb, ku, _ = q.shape
    r, c = np.arange(rows)[:, None], np.arange(cols)[None]
    b, g, half = r // 16, r % 8, (r % 16) // 8
    h, t, j, p, e = (c % 64) // 32, (c % 32) // 8, (c % 8) // 4, (c % 4) // 2, c % 2
    byte = q[:, :, b, c // 64, 16 * (4 * g + t) + 4 * (2 * h + j) + 2 * e + p]
    code = np.where(half == 0, byte & 15, byte >> 4).astype(np.float64)
    return (code - 8) * scale[:, :, b, c // group, g, half]


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def swiglu(gate, up, clamp):
    if clamp > 0:
        gate, up = np.clip(gate, -clamp, clamp), np.clip(up, -clamp, clamp)
    return silu(gate) * up


def balance(z, ids, mask, E, k, alpha, sigmoid):
    """loss, counts, P, dlogits (gradient 1) of the valid tokens."""
    N = z.shape[0]
    live = np.ones(N, bool) if mask is None else mask != 0
    T = max(1, int(live.sum()))
    counts = np.bincount(ids[live].ravel(), minlength=E)
    f = counts / (T * k)
    zl = z[live]
    if sigmoid:
        a = 1 / (1 + np.exp(-zl))
        u = 1 - a
    else:
        m = zl.max(1, keepdims=True) if zl.size else np.zeros((0, 1))
        a = np.exp(zl - np.where(np.isfinite(m), m, 0))
        u = np.ones_like(a)
    tot = a.sum(1, keepdims=True)
    p = np.divide(a, tot, out=np.zeros_like(a), where=tot > 0)
    P = p.sum(0) / T
    d = np.zeros((N, E))
    d[live] = alpha * E / T * p * u * (f - (p * f).sum(1, keepdims=True))
    mag = np.zeros((N, E))  # sum of the magnitudes that the gradient is the difference of
    f0 = np.abs(f - 1 / E)
    mag[live] = alpha * E / T * p * u * (f0 + (p * f0).sum(1, keepdims=True))
    return alpha * E * (f * P).sum(), counts, P, d, mag

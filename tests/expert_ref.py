"""Plain 64-bit statements of the operators in include/tk_expert.h (numpy), and
what their tests share."""
import numpy as np

import layer_ref as ref

E4M3 = ref.e4m3_values()


def spans(offsets, n):
    """(first, last) row of each expert: offsets inside 0 .. n, none below the one before it."""
    if offsets is None:
        return [(0, n)]
    out = []
    for a, b in zip(offsets[:-1], offsets[1:]):
        lo = min(max(int(a), 0), n)
        out.append((lo, min(max(int(b), lo), n)))
    return out


def take(x, index, lo, hi):
    """Rows lo .. hi - 1 of x by the index; zeros for one that names no row."""
    if index is None:
        return x[lo:hi]
    i = index[lo:hi].astype(np.int64)
    ok = (i >= 0) & (i < len(x))
    return np.where(ok[:, None], x[np.where(ok, i, 0)] if len(x) else 0.0, 0.0)


def gemm(x, index, offsets, n, w, start):
    """(out, sum of the terms' magnitudes); `start`: what rows of no expert keep."""
    out, mag = start.astype(np.float64), np.zeros(start.shape)
    for e, (lo, hi) in enumerate(spans(offsets, n)):
        rows = take(x, index, lo, hi)
        out[lo:hi], mag[lo:hi] = rows @ w[e].T, np.abs(rows) @ np.abs(w[e]).T
    return out, mag


def dgrad(dy, index, offsets, n, w, start):
    return gemm(dy, index, offsets, n, np.swapaxes(w, 1, 2), start)


def wgrad(dy, dy_index, x, x_index, offsets, n, start):
    """start + the sums, and their terms' magnitudes."""
    out, mag = start.astype(np.float64), np.abs(start.astype(np.float64))
    for e, (lo, hi) in enumerate(spans(offsets, n)):
        a, b = take(dy, dy_index, lo, hi), take(x, x_index, lo, hi)
        out[e] += a.T @ b
        mag[e] += np.abs(a).T @ np.abs(b)
    return out, mag


def coded(codes, scales, u8, fp4=False):
    """The values of codes [rows, columns (/2)] with row-major scales [rows, groups]."""
    if fp4:
        v = np.empty((codes.shape[0], codes.shape[1] * 2))
        v[:, 0::2], v[:, 1::2] = ref.E2M1[codes & 15], ref.E2M1[codes >> 4]
    else:
        v = E4M3[codes]
    s = ref.e8m0_value(scales) if u8 else scales.astype(np.float64)
    return v * np.repeat(s, v.shape[1] // s.shape[1], axis=1)


def swiglu(h, weight, clamp):
    """(y, pieces) of packed h = g | u in 64 bits."""
    h = h.astype(np.float64)
    half = h.shape[1] // 2
    g, u = h[:, :half], h[:, half:]
    gc, uc = np.minimum(g, clamp), np.clip(u, -clamp, clamp)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-gc))
    w = 1.0 if weight is None else weight.astype(np.float64)[:, None]
    return gc * s * uc * w, (g, u, gc, uc, s, w)


def swiglu_backward(dy, h, weight, clamp):
    """dh, dweight, y and the magnitude of dweight's terms."""
    y, (g, u, gc, uc, s, w) = swiglu(h, weight, clamp)
    dy, a = dy.astype(np.float64), gc * s
    dg = np.where(g <= clamp, dy * w * uc * (s + a * (1 - s)), 0.0)
    du = np.where(np.abs(u) <= clamp, dy * w * a, 0.0)
    return np.concatenate([dg, du], 1), (dy * a * uc).sum(1), y, np.abs(dy * a * uc).sum(1)

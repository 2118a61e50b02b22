"""Plain 64-bit statements of the operators in include/tk_layer.h (numpy), and
the bit-level helpers their tests share."""
import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
UB16 = 2.0 ** -8   # half a step of bf16
UE4M3 = 2.0 ** -4  # half a step of E4M3
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def bf16_bits(x):
    """fp32 -> bf16 bits, nearest even (finite values and infinities; NaN stays NaN)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32)


def round_bf16(x):
    return bf16_value(bf16_bits(x))


def e4m3_values():
    """The value of every E4M3 byte (0x7F and 0xFF are NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def e8m0_value(b):
    b = np.asarray(b).astype(np.float64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127))


# ---- norm ---------------------------------------------------------------------------------------


def norm_stream(x, residual, bf16):
    """h: the stream with the residual added, as it is stored (fp32 values)."""
    if residual is None:
        return x.astype(np.float32)
    h = x.astype(np.float32) + residual.astype(np.float32)
    return round_bf16(h) if bf16 else h


def norm(h, weight, eps):
    """(rstd, y) in 64 bits."""
    h = h.astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt(np.square(h).sum(1) / h.shape[1] + float(np.float32(eps)))
        return rstd, h * rstd[:, None] * weight.astype(np.float64)


def norm_backward(dy, h, weight, rstd, dres):
    dy, h, w, r = (np.asarray(a, dtype=np.float64) for a in (dy, h, weight, rstd))
    a = h * r[:, None]
    g = dy * w
    dx = r[:, None] * (g - a * (g * a).sum(1, keepdims=True) / h.shape[1])
    if dres is not None:
        dx = dx + dres.astype(np.float64)
    return dx, (dy * a).sum(0)


# ---- routing ------------------------------------------------------------------------------------


def scores(logits, softmax):
    x = logits.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if not softmax:
            t = np.exp(-np.abs(x))
            return np.where(x >= 0, 1 / (1 + t), t / (1 + t))
        top = x.max(1, keepdims=True)
        e = np.exp(x - np.where(top == -np.inf, 0, top))
        s = e.sum(1, keepdims=True)
        return e / np.where(s == 0, 1, s)


def route(logits, bias, k, n_group, topk_group, softmax, normalise, scale):
    """Token by token, pick by pick, from the definition.  Returns (idx, weight in 64 bits)."""
    T, E = logits.shape
    s = scores(logits, softmax)
    idx, w = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    per = E // n_group
    for t in range(T):
        x = logits[t].astype(np.float32)
        key = x.copy()
        if bias is not None or n_group > 1:
            with np.errstate(over="ignore"):
                key = s[t].astype(np.float32)
                if bias is not None:
                    key = key + bias.astype(np.float32)
        live = (x != -np.inf) & (key != -np.inf)
        if np.isnan(x).any() or np.isnan(key).any() or (softmax and (x == np.inf).any()):
            idx[t], w[t] = np.arange(k), np.nan
            continue
        if n_group > 1:
            value = []
            for g in range(n_group):
                m = np.sort(key[g * per:(g + 1) * per][live[g * per:(g + 1) * per]])[::-1]
                value.append(-np.inf if len(m) == 0 else m[0] if len(m) == 1 else np.float32(m[0] + m[1]))
            kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            live &= np.isin(np.arange(E) // per, kept)
        order = sorted(np.flatnonzero(live), key=lambda e: (-key[e], e))[:k]
        idx[t, :len(order)] = order
        ws = s[t, order]
        if normalise and ws.sum() != 0:
            ws = ws / ws.sum()
        w[t, :len(order)] = ws * float(np.float32(scale))
    return idx, w


def route_backward(dweight, idx, logits, softmax, normalise, scale):
    """The gradient, and the sum over its terms' magnitudes (what an fp32 evaluation's error grows with)."""
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        chosen, d = [], np.zeros(E)
        for j, e in enumerate(idx[t]):
            if 0 <= e < E and e not in chosen:
                chosen.append(int(e))
                d[e] = float(np.float32(scale)) * float(dweight[t, j])
        c = np.zeros(E)
        c[chosen] = 1
        s = scores(logits[t:t + 1], softmax)[0]
        if softmax:
            if normalise:
                x = np.where(c > 0, logits[t].astype(np.float64), -np.inf)
                s = scores(x[None], True)[0]
            dot = (d * s).sum()
            out[t] = s * (d - dot)
            mag[t] = s * (np.abs(d) + (np.abs(d) * s).sum())
        else:
            slope = scores(-logits[t:t + 1], False)[0]
            if normalise and (s * c).sum() != 0:
                s = s * c / (s * c).sum()
                out[t] = s * slope * (d - (d * s).sum()) * c
                mag[t] = s * slope * (np.abs(d) + np.abs(d * s).sum()) * c
            else:
                out[t] = d * s * slope * c
                mag[t] = np.abs(out[t])
    return out, mag


# ---- products -----------------------------------------------------------------------------------


def fp4_values(codes, scales, u8):
    """codes uint8 [..., in/2], scales [..., groups] -> 64-bit weights [..., in]."""
    w = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], -1)
    sc = e8m0_value(scales) if u8 else scales.astype(np.float64)
    return (w.reshape(*sc.shape, -1) * sc[..., None]).reshape(w.shape)


def x_values(x, x_scales, kind):
    """kind: bf16 (bits), fp8 (codes with fp32 scales), fp8e (codes with UE8M0 scales)."""
    if kind == "bf16":
        return bf16_value(x).astype(np.float64)
    v = e4m3_values()[x]
    sc = e8m0_value(x_scales) if kind == "fp8e" else x_scales.astype(np.float64)
    return (v.reshape(*sc.shape, -1) * sc[..., None]).reshape(v.shape)


def gemv(xv, idx, k, slots, wv):
    """(out, sum of the products' magnitudes), rows tokens*k."""
    rows = idx.size
    out, mag = np.zeros((rows, wv.shape[1])), np.zeros((rows, wv.shape[1]))
    for r, e in enumerate(idx.reshape(-1)):
        if 0 <= e < wv.shape[0]:
            v = xv[r if slots else r // k]
            out[r] = wv[e] @ v
            mag[r] = np.abs(wv[e]) @ np.abs(v)
    return out, mag

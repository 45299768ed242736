"""Plain 64-bit forms of the routing operators and of the 4-bit expert
products, written from their definitions with numpy, token by token."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def choose(logits, k, G=1, KG=1, bias=None, valid=None):
    """int32 [T, k]: ids by descending key, -1 where too few experts are on."""
    T, E = logits.shape
    with np.errstate(over="ignore", invalid="ignore"):
        key = logits.astype(np.float32)
        if bias is not None:
            key = key + bias.astype(np.float32)[None]
    out = np.full((T, k), -1, np.int32)
    low = -float(np.finfo(np.float32).max)
    gs = E // G
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        on = np.isfinite(logits[t]) & np.isfinite(key[t])
        if G > 1:
            score = []
            for g in range(G):
                own = sorted((float(key[t, e]) if on[e] else low for e in range(g * gs, g * gs + gs)),
                             reverse=True)
                score.append(own[0] + own[1] if gs > 1 else own[0])
            keep = sorted(range(G), key=lambda g: (-score[g], g))[:KG]
            for g in range(G):
                if g not in keep:
                    on[g * gs:(g + 1) * gs] = False
        ids = sorted(np.flatnonzero(on), key=lambda e: (-float(key[t, e]), e))[:k]
        out[t, :len(ids)] = ids
    return out


def _log_z(x, score):
    return x if score == 0 else -np.logaddexp(0.0, -x)


def probs(logits, score, valid=None):
    x = logits.astype(np.float64)
    on = np.isfinite(x)
    if valid is not None:
        on &= (np.asarray(valid) != 0)[:, None]
    l = np.where(on, _log_z(np.where(on, x, 0.0), score), -np.inf)
    m = l.max(1, keepdims=True)
    z = np.where(on, np.exp(np.where(on, l - np.where(np.isfinite(m), m, 0), 0)), 0.0)
    s = z.sum(1, keepdims=True)
    return z / np.where(s > 0, s, 1)


def present(logits, idx, valid=None):
    T, E = logits.shape
    ok = (idx >= 0) & (idx < E)
    x = np.take_along_axis(logits.astype(np.float64), np.where(ok, idx, 0), 1)
    ok &= np.isfinite(x)
    if valid is not None:
        ok &= (np.asarray(valid) != 0)[:, None]
    return np.where(ok, x, 0.0), ok


def weights(logits, idx, score, normalize, scale=1.0, valid=None):
    x, ok = present(logits, idx, valid)
    if normalize:
        l = np.where(ok, _log_z(x, score), -np.inf)
        m = l.max(1, keepdims=True)
        z = np.where(ok, np.exp(np.where(ok, l - np.where(np.isfinite(m), m, 0), 0)), 0.0)
        s = z.sum(1, keepdims=True)
        w = z / np.where(s > 0, s, 1)
    elif score == 1:
        w = np.where(ok, np.exp(_log_z(x, 1)), 0.0)
    else:
        p = probs(logits, 0, valid)
        w = np.where(ok, np.take_along_axis(p, np.where(ok, idx, 0), 1), 0.0)
    return scale * w


def counts(idx, E, B, valid=None):
    T, k = idx.shape
    c = np.zeros((B, E), np.int32)
    n = np.zeros(B, np.int32)
    L = T // B if B else 0
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        n[t // L] += 1
        for e in idx[t]:
            if 0 <= e < E:
                c[t // L, e] += 1
    return c, n


def balance(logits, idx, score, coef, B, valid=None):
    T, E = logits.shape
    k = idx.shape[1]
    c, n = counts(idx, E, B, valid)
    p = probs(logits, score, valid).reshape(B, -1, E)
    m = np.maximum(n, 1)[:, None]
    mean = p.sum(1) / m
    loss = coef / B * float((E / (k * m) * c * mean).sum())
    return c, mean, n, loss


def gradient(logits, idx, score, normalize, scale=1.0, dw=None, coef=0.0, c=None, n=None,
             dloss=None, valid=None):
    """Gradient of the logits, and the sum of the magnitudes of its terms."""
    T, E = logits.shape
    k = idx.shape[1]
    x = logits.astype(np.float64)
    on = np.isfinite(x)
    if valid is not None:
        on &= (np.asarray(valid) != 0)[:, None]
    xs = np.where(on, x, 0.0)
    slope = np.exp(-np.logaddexp(0.0, xs)) if score else np.ones_like(xs)
    dx = np.zeros((T, E))
    size = np.zeros((T, E))
    if dloss is not None:
        B = len(n)
        m = np.maximum(n, 1).astype(np.float64)[:, None]
        a = coef * dloss * E / (B * k) * (c - c[:, :1]) / (m * m)
        a = np.repeat(a, T // B, 0)
        p = probs(logits, score, valid)
        dot = (a * p).sum(1, keepdims=True)
        dx += p * (a - dot) * slope
        size += p * (np.abs(a) + (np.abs(a) * p).sum(1, keepdims=True)) * slope
    if dw is not None:
        xe, ok = present(logits, idx, valid)
        g = np.where(ok, dw.astype(np.float64) * scale, 0.0)
        w = weights(logits, idx, score, normalize, 1.0, valid)
        neg = np.exp(-np.logaddexp(0.0, xe)) if score else np.ones_like(xe)
        gw = (g * w).sum(1, keepdims=True)
        ga = (np.abs(g) * w).sum(1, keepdims=True)
        if normalize:
            d, s = w * (g - gw) * neg, w * (np.abs(g) + ga) * neg
        else:
            d, s = w * g * neg, w * np.abs(g) * neg
            if score == 0:
                p = probs(logits, 0, valid)
                dx -= p * gw
                size += p * ga
        for t in range(T):
            for j in range(k):
                if ok[t, j]:
                    dx[t, idx[t, j]] += d[t, j]
                    size[t, idx[t, j]] += s[t, j]
    return np.where(on, dx, 0.0), np.where(on, size, 0.0)


def decode_w4(codes, scales):
    """float64 [.., K] from uint8 codes [.., K / 2] and scale bytes [.., K / 32]."""
    q = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), np.uint8)
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    v = E2M1[q & 7] * np.where(q & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int32) - 127))
    return v * np.repeat(s, 32, -1)


def products(x, codes, scales, gated):
    """Outputs of rows x (float64 [m, K]) of one expert, and a bound on the
    effect of one fp32 rounding (2^-24) of each product on each output."""
    w = decode_w4(codes, scales)
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if not gated:
        return y, mag
    N = y.shape[1] // 2
    g, u = y[:, :N], y[:, N:]
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    # |d silu / dg| <= 1.1; 8 more roundings inside the activation
    return s * u, 1.1 * mag[:, :N] * np.abs(u) + np.abs(s) * mag[:, N:] + 8 * np.abs(s * u)

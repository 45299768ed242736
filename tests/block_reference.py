"""Plain 64-bit forms of layer norm, of dropout in the combine and of the 8-bit
integer products, written from their definitions with numpy."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    """Half a step of the output type, relative."""
    return {"bf16": 2.0 ** -8, "fp32": U}[dtype]


# ------------------------------------------------------------------ layer norm

def norm(x, w, b, eps):
    m = x.mean(1, keepdims=True)
    d = x - m
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return d * r * w + b, m[:, 0], r[:, 0]


ROW_ADDS = 128  # most additions that a channel passes on the way into a row's sum: 64
#                 channels of a lane, 6 steps in a wave, 16 waves, and some to spare


def norm_bounds(x, w, b, eps, dtype):
    """Largest errors of y, mean and rstd: each sum rounds at most ROW_ADDS times."""
    y, m, r = norm(x, w, b, eps)
    d = np.abs(x - m[:, None])
    em = ROW_ADDS * U * np.abs(x).mean(1, keepdims=True)
    ed = em + U * d + U * em
    var = (d * d).mean(1, keepdims=True)
    ev = 2 * (d * ed).mean(1, keepdims=True) + (ed * ed).mean(1, keepdims=True) + ROW_ADDS * U * var
    er = 0.5 * ev / (var + eps) * 1.1 + 6 * U          # relative
    t = np.abs(w) * r[:, None]
    ey = t * ed + t * d * (er + 3 * U) + 2 * U * (t * d + np.abs(b)) + half_step(dtype) * np.abs(y)
    return ey * 1.01 + 2.0 ** -133, em[:, 0], (er * r[:, None])[:, 0]


def norm_grad(x, dy, w, m, r, skip=None):
    n = (x - m[:, None]) * r[:, None]
    a = dy * w
    dx = r[:, None] * (a - a.mean(1, keepdims=True) - n * (a * n).mean(1, keepdims=True))
    if skip is not None:
        dx = dx + skip
    return dx, (dy * n).sum(0), dy.sum(0)


def norm_grad_bounds(x, dy, w, m, r, skip, x_dtype, w_dtype):
    n = np.abs((x - m[:, None]) * r[:, None])
    a = np.abs(dy * w)
    c1, c2 = a.mean(1, keepdims=True), (a * n).mean(1, keepdims=True)
    e = a * U + ROW_ADDS * U * c1 + n * ROW_ADDS * U * c2 + 2 * U * n * c2 + 4 * U * (a + c1 + n * c2)
    dx, dw, db = norm_grad(x, dy, w, m, r, skip)
    edx = r[:, None] * e * 1.01 + (2 * U + half_step(x_dtype)) * np.abs(dx) + 2.0 ** -133
    if skip is not None:
        edx = edx + U * np.abs(skip)
    # a run of T / 256 rows, then joins of fewer than 64
    adds = len(x) / 256 + 64
    ew = (adds + 3) * U * np.abs(dy * n).sum(0) + half_step(w_dtype) * np.abs(dw) + 2.0 ** -133
    eb = adds * U * np.abs(dy).sum(0) + half_step(w_dtype) * np.abs(db) + 2.0 ** -133
    return edx, ew, eb


# --------------------------------------------------------------------- dropout

def philox(counter, key):
    """Words [..., 4] of Philox4x32 with ten rounds at counters [..., 4]."""
    c = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ np.uint64(k0), q & low, (p >> half) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1).astype(np.uint32)


def kept(T, H, p, seed, offset):
    """bool [T, H]."""
    seed, offset = int(seed) % 2 ** 64, int(offset) % 2 ** 64
    n = (H + 3) // 4
    ctr = np.empty((T, n, 4), np.uint64)
    ctr[..., 0] = np.arange(n)[None]
    ctr[..., 1] = np.arange(T)[:, None]
    ctr[..., 2], ctr[..., 3] = offset & 0xFFFFFFFF, offset >> 32
    words = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(T, 4 * n)[:, :H]
    return words >= min(int(np.rint(p * 2.0 ** 32)), 2 ** 32 - 1)


def combine(eo, slot, w, keep, p, residual=None):
    """(y, bound of its error): k fused steps, the factor, the skip, one rounding to bf16."""
    T, k = slot.shape
    s, mag = np.zeros((T, eo.shape[1])), np.zeros((T, eo.shape[1]))
    for t in range(T):
        for j in range(k):
            if slot[t, j] >= 0:
                v = w[t, j] * eo[slot[t, j]]
                s[t] += v
                mag[t] += np.abs(v)
    f = 1 / (1 - p)
    y = np.where(keep, s * f, 0.0)
    e = np.where(keep, (k + 3) * U * mag * f, 0.0)
    if residual is not None:
        y = y + residual
    return y, e + (2 * U + 2.0 ** -8) * np.abs(y) + 2.0 ** -133


DOT_ADDS = 128  # of a dot product over a row: 64 channels of a lane, 6 steps, 16 waves


def combine_grad(dy, eo, slot, w, keep, p):
    """(d_expert_out by slot as {slot: row}, its bounds, d_weights, its bounds)."""
    g = np.where(keep, dy / (1 - p), 0.0)
    T, k = slot.shape
    rows, bounds = {}, {}
    dw, ew = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            s = int(slot[t, j])
            if s < 0:
                continue
            rows[s] = w[t, j] * g[t]
            bounds[s] = (4 * U + 2.0 ** -8) * np.abs(rows[s]) + 2.0 ** -133
            dw[t, j] = (g[t] * eo[s]).sum()
            ew[t, j] = (DOT_ADDS + 3) * U * np.abs(g[t] * eo[s]).sum() + 2.0 ** -140
    return rows, bounds, dw, ew


# --------------------------------------------------------- 8-bit integer rows

def quant(x):
    """int8 codes and fp32 scales of fp32-representable rows, to the bit."""
    x = x.astype(np.float32)
    scale = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / scale[:, None])
    return np.where(scale[:, None] > 0, q, 0).astype(np.int8), scale


def i8_products(q, row_scale, w, scale, gated):
    """(y, bound) of rows q int8 [M, K] with weights int8 [n2, K]."""
    s = q.astype(np.float64) @ w.astype(np.float64).T  # whole numbers below 2^53: exact
    y = s * row_scale.astype(np.float64)[:, None] * scale.astype(np.float64)[None]
    e = 4 * U * np.abs(y)
    if gated:
        n = y.shape[1] // 2
        g, up = y[:, :n], y[:, n:]
        sg = g / (1 + np.exp(-g))
        # exp's argument is off by 4 U |g|, the exponential by a few steps, then a sum,
        # a quotient and a product
        e = np.abs(sg * up) * (12 + 5 * np.abs(g)) * U
        y = sg * up
    return y, e + 2.0 ** -8 * np.abs(y) + 2.0 ** -133

"""The block-scaled 8-bit-float operators from their formulas, in numpy: codes
and their values from the bit layout, sums in 64 bits.  Shares nothing with
the library."""
import numpy as np

B = 128
TINY = np.float32(2.0 ** -126)


def _value(c):
    sign = -1.0 if c & 0x80 else 1.0
    e, m = (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return np.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


VALUES = np.array([_value(c) for c in range(256)])
POSITIVE = VALUES[:127]                       # codes 0 .. 126: 0 .. 448, rising


def encode(v):
    """Codes of float32 values: nearest, ties to the even code, saturating; NaN -> 0x7f."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(v, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.searchsorted(POSITIVE, a).clip(1, 126)
    lo = hi - 1
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(a == 0, 0, c)
    c = np.where(np.signbit(v), c | 0x80, c)
    return np.where(np.isnan(v), 0x7f, c).astype(np.uint8)


def quantize(x):
    """(codes uint8 [M, K], scales float32 [M, kb]) of x [M, K]."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    kb = -(-K // B)
    codes, s = np.zeros((M, K), np.uint8), np.zeros((M, kb), np.float32)
    with np.errstate(all="ignore"):
        for b in range(kb):
            t = x[:, b * B:(b + 1) * B]
            s[:, b] = np.maximum(np.abs(t).max(axis=1) / np.float32(448), TINY)
            inv = np.float32(1) / s[:, b]
            codes[:, b * B:(b + 1) * B] = encode(t * inv[:, None])
    return codes, s


def expand(S, N, K):
    """Scales [nb, kb] at every element of an [N, K] matrix, 64 bits."""
    return np.repeat(np.repeat(np.asarray(S, np.float64), B, 0)[:N], B, 1)[:, :K]


def dense(codes, S):
    return VALUES[codes] * expand(S, *codes.shape)


def rounded(x):
    """x as the values of its codes."""
    c, s = quantize(x)
    return VALUES[c] * np.repeat(s.astype(np.float64), B, 1)[:, :c.shape[1]]


def product(W, S, x):
    """(y, A): x rounded to codes, times W; A the sum of absolute terms."""
    w, xv = dense(W, S), rounded(x)
    with np.errstate(all="ignore"):
        return xv @ w.T, np.abs(xv) @ np.abs(w).T


def bound(K, A):
    """Of the fp32 arithmetic: 128 additions of exact products per block at 2^-23 of the block's absolute sum each
    (whatever their order, truncated or rounded), then three roundings of scale and product and one addition per
    block at 2^-24."""
    kb = -(-K // B)
    return (128 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * A + 1e-37


#: relative half-ulp and half of the smallest step of the result types
ROUND = {"float32": (2.0 ** -24, 2.0 ** -150), "float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}


def out_bound(y, e, dtype):
    rel, least = ROUND[dtype]
    return e + rel * (np.abs(y) + e) + least


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def gated(Wg, Sg, Wu, Su, x):
    """(h, e): the gated pair before its rounding, and how far fp32 arithmetic may be off."""
    K = Wg.shape[1]
    g, Ag = product(Wg, Sg, x)
    u, Au = product(Wu, Su, x)
    eg, eu = bound(K, Ag), bound(K, Au)
    h = silu(g) * u
    # |silu'| < 1.1; exp, the division and the product in fp32: 2^-21 of the result
    return h, 1.1 * np.abs(u) * eg + np.abs(silu(g)) * eu + 1.1 * eg * eu + 2.0 ** -21 * np.abs(h)


def down_product(W, S, h, e):
    """(y, bound) of W times the rounded h when h is known to +-e: codes whose value lies within the uncertainty of a
    boundary may be the next one, and a scale moves with its block's largest |h|."""
    R, K = h.shape
    kb = -(-K // B)
    hv, he = np.zeros_like(h), np.zeros_like(h)
    with np.errstate(all="ignore"):
        c, s = quantize(h.astype(np.float32))
    for b in range(kb):
        k = slice(b * B, min((b + 1) * B, K))
        sb = s[:, b:b + 1].astype(np.float64)
        drift = (e[:, k].max(axis=1, keepdims=True) / 448 + 2.0 ** -22 * sb) / sb   # relative error of the scale
        v = np.abs(h[:, k]) / sb
        dv = e[:, k] / sb + v * (drift + 2.0 ** -22)
        lo = VALUES[encode(np.maximum(v - dv, 0.0))]
        hi = VALUES[encode(v + dv)]
        q = VALUES[c[:, k]]
        hv[:, k] = q * sb
        he[:, k] = np.maximum(np.abs(hi - np.abs(q)), np.abs(np.abs(q) - lo)) * sb * (1 + drift) + np.abs(q) * sb * drift
    w = dense(W, S)
    A = (np.abs(hv) + he) @ np.abs(w).T
    return hv @ w.T, bound(K, A) + he @ np.abs(w).T


def route(x, k, score, normalize, factor=1.0):
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    T, E = x.shape
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(x, order, 1)
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = np.where(v[:, :1] == -np.inf, 0.0, v[:, :1])
            w = np.exp(v - m)
            total = w.sum(1, keepdims=True) if normalize else np.exp(x - m).sum(1, keepdims=True)
        else:
            w = 1 / (1 + np.exp(-v))
            total = w.sum(1, keepdims=True) if normalize else np.ones((T, 1))
        w = np.where(total != 0, w / total, 0.0) * factor
    flat = order.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    slots = np.empty(T * k, np.int64)
    slots[perm] = np.arange(T * k)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return w, order, offsets, perm // k, slots.reshape(T, k)


def weights(rng, N, K):
    """Codes and scales as a checkpoint holds them: normal weights, each block scaled to the largest code."""
    nb, kb = -(-N // B), -(-K // B)
    w = (rng.standard_normal((N, K)) / np.sqrt(max(K, 1))).astype(np.float32)
    S = np.zeros((nb, kb), np.float32)
    for i in range(nb):
        for j in range(kb):
            S[i, j] = np.abs(w[i * B:(i + 1) * B, j * B:(j + 1) * B]).max() / 448
    return encode(w / expand(S, N, K)), S

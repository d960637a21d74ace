"""The position rotation, the paged cache and the attention over it in 64 bits with numpy, and how far a result may be
from them."""
import numpy as np

EPS = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}  # half a step, relative
TINY = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}  # half the smallest step
LEAST = 2.0 ** -100
TOP = 448.0


def _values():
    """The 256 e4m3 values: sign, four exponent bits (bias 7), three mantissa bits; 0x7f and 0xff are NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = -a if c >> 7 else a
    return v


VALUES = _values()


def codes_of(x):
    """x in 64 bits to the nearest code, ties to even; what is not finite to a NaN code."""
    a = np.abs(x)
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.floor(np.log2(np.where(np.isfinite(a) & (a >= 2.0 ** -6), a, 2.0 ** -6)))
        step = 2.0 ** (e - 3)
        r = np.rint(a / step) * step
        r = np.minimum(r, TOP)
        e = np.floor(np.log2(np.where(np.isfinite(r) & (r >= 2.0 ** -6), r, 2.0 ** -6)))
        sub = r < 2.0 ** -6
        c = np.where(sub, np.rint(r * 512), (e + 7) * 8 + np.rint((r / 2.0 ** e - 1) * 8))
    c = np.where(np.isfinite(x), c, 127).astype(np.uint8)
    return c | np.where(np.signbit(x), 128, 0).astype(np.uint8)


def frequencies(rot, base=10000.0, scaling=None, scale=1.0, original=0.0, low=1.0, high=4.0):
    i = np.arange(rot // 2)
    if scaling == "ntk":
        base = base * scale ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / scale
    if scaling == "parts":
        k = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        return f * k + f / scale * (1 - k)
    return f


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rope(x, positions, f, interleaved=False, inverse=False, factor=1.0):
    """x [T, heads, dim] turned, and how far a result may be: 2^-21 factor (|a| + |b|) for both values of a pair."""
    x = np.asarray(x, np.float64)
    y, e = x.copy(), np.zeros_like(x)
    first, second = pairs(2 * len(f), interleaved)
    w = np.asarray(positions, np.float64)[:, None] * f[None, :]
    c, s = np.cos(w)[:, None], np.sin(w)[:, None] * (-1 if inverse else 1)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = factor * (a * c - b * s), factor * (b * c + a * s)
    e[..., first] = e[..., second] = 2.0 ** -21 * abs(factor) * (np.abs(a) + np.abs(b))
    return y, e


def rounded(y, e, dtype):
    """The bound of a value within e of y that was then rounded to dtype."""
    return e + EPS[dtype] * (np.abs(y) + e) + TINY[dtype]


def need(top):
    """The smallest power of two at which top (the largest finite value) is at most 448 of it."""
    top = np.asarray(top, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.ceil(np.log2(top / TOP)), -100)
    e = np.where(top > TOP * 2.0 ** e, e + 1, e)
    e = np.where(top <= TOP * 2.0 ** (e - 1), e - 1, e)
    return 2.0 ** np.maximum(e, -100)


class Batch:
    """Sequences of given lengths whose last rows are new, and their pages in a random order."""

    def __init__(self, rng, new, lengths, page, spare=2, width=0):
        self.new, self.lengths, self.page = list(new), list(lengths), page
        counts = [-(-n // page) for n in lengths]
        self.pages = sum(counts) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(new), max([width] + counts)), -7, np.int32)  # (never looked at behind a sequence)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.offsets[-1])

    def positions(self):
        return np.concatenate([np.arange(n - m, n) for m, n in zip(self.new, self.lengths)] + [np.zeros(0, np.int64)])


def append(codes, scales, x, batch):
    """codes [pages, heads, page, dim] and scales after the rows x [T, heads, dim] (64 bits) went in."""
    codes, scales = codes.copy(), scales.astype(np.float64).copy()
    P = batch.page
    for b, (m, n) in enumerate(zip(batch.new, batch.lengths)):
        at, pos = batch.offsets[b], n - m
        while pos < n:
            p, slot = batch.table[b, pos // P], pos % P
            rows = min(P - slot, n - pos)
            v = x[at:at + rows].transpose(1, 0, 2)
            a = np.abs(v)
            top = np.where(np.isfinite(a), a, 0).max(axis=(1, 2))
            s = need(top)
            if slot:
                s = np.maximum(s, scales[p])
                grown = s != scales[p]
                old = VALUES[codes[p, :, :slot]] * (scales[p] / s)[:, None, None]
                codes[p, :, :slot] = np.where(grown[:, None, None], codes_of(old), codes[p, :, :slot])
            codes[p, :, slot:slot + rows] = codes_of(v / s[:, None, None])
            scales[p] = s
            pos, at = pos + rows, at + rows
    return codes, scales


def attention(q, k, ks, v, vs, batch, scale, causal=True, window=0, small=False):
    """(y, lse, bound of y before its rounding, bound of lse) in 64 bits; q [T, query heads, dim] as the values it holds,
    fp32 queries (u32) or 16-bit ones.  small: some 16-bit values are below 2^-13 of their head's largest, m, and may be
    off by 2^-21 m.  A score is then off by at most d = |scale| 2^-21 m sum |k_ji|, and p_j / sum p by exp(2 d) - 1 of it."""
    T, Hq, D = q.shape
    H, P = k.shape[1], batch.page
    y, e = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, le = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b, (m, n) in enumerate(zip(batch.new, batch.lengths)):
        ids = batch.table[b, :-(-n // P)]
        if n == 0:
            continue
        K = (VALUES[k[ids]] * ks[ids][:, :, None, None]).transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
        V = (VALUES[v[ids]] * vs[ids][:, :, None, None]).transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
        pos = np.arange(n - m, n)[:, None]
        j = np.arange(n)[None, :]
        seen = np.ones((m, n), bool)
        if causal:
            seen = j <= pos
            if window:
                seen &= j > pos - window
        rows = slice(batch.offsets[b], batch.offsets[b + 1])
        for h in range(Hq):
            g = h // (Hq // H)
            with np.errstate(invalid="ignore", over="ignore"):
                x = np.where(seen, scale * (q[rows, h] @ K[g].T), -np.inf)
                X = np.where(seen, abs(scale) * (np.abs(q[rows, h]) @ np.abs(K[g]).T), 0).max(axis=1)
            top = x.max(axis=1)
            some = top > -np.inf
            w = np.where(seen, np.exp(x - np.where(some, top, 0)[:, None]), 0)
            total = w.sum(axis=1)
            with np.errstate(invalid="ignore", divide="ignore"):
                r = np.where(some[:, None], (w @ V[g]) / total[:, None], 0)
                spread = np.where(some[:, None], (w @ np.abs(V[g])) / total[:, None], 0)
                lse[rows, h] = np.where(some, top + np.log(total), -np.inf)
            c = (seen.sum(axis=1) + D + 64) * 2.0 ** -22 * (1 + X)
            if small and q.dtype != np.float32:
                d = abs(scale) * 2.0 ** -21 * np.abs(q[rows, h]).max(axis=1) * np.where(seen, np.abs(K[g]).sum(axis=1), 0).max(axis=1)
                c = c + np.expm1(2 * d)
            y[rows, h], e[rows, h] = r, c[:, None] * spread
            le[rows, h] = c + 2.0 ** -22 * np.where(some, np.abs(lse[rows, h]), 0)
            e[rows, h] += 2.0 ** -11 * spread if q.dtype != np.float32 else 2.0 ** -20 * spread
    return y, lse, e, le

"""Attention over the paged cache at its limits, on every kernel that a call may go to: scales that differ from group to
group, windows near 2^31, values far apart, NaN codes in tiles that masks cut, long sequences of which no tile may be
lost."""
import math

import numpy as np
import pytest

import kv_reference as R
from test_gpu_kv import _as, _cache, _np, _t, _u8, _within

pytestmark = pytest.mark.gpu

# rows of a sequence, table width (0: as needed) and type that lead to each kernel with 2 cache heads and a group of 4
# (kv_attention.cu: up to 32 rows; 9 to 32 16-bit ones of tables of many pages; more; more fp32 ones)
KERNELS = {"few": ("bfloat16", 2, 0), "few fp32": ("float32", 3, 0), "slim": ("float16", 5, 1300), "slim bf16": ("bfloat16", 8, 1300),
           "tc": ("bfloat16", 70, 0), "tc fp16": ("float16", 70, 0), "rows": ("float32", 40, 0)}


def _i32(a):
    return _t(np.asarray(a, np.int32))


def _run(q, cache, x, batch, **k):
    y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _i32(batch.lengths), offsets=_t(batch.offsets), lse=True, **k)
    assert q.qmm_device_status() == 0
    return y, lse


@pytest.mark.parametrize("kernel", [k for k in KERNELS if not k.startswith("tc")])
def test_every_group_of_tokens_has_the_scale_of_its_page(cuda_lib, kernel):
    """Pages of 16 tokens whose scales differ by up to 2^40, in short sequences (a tile's scales are read as soon as its
    codes are there): against 64 bits, and the same bits again and again."""
    import torch
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    rng = np.random.default_rng(70)
    lengths = [max(n, new) for n in (130, 90, 300, 17, 500, 64)]
    batch = R.Batch(rng, [new] * 6, lengths, 16, width=width)
    cache, codes, scales = _cache(q, rng, batch, 2, 64, spread=20)
    x, xv = _as(2.0 ** -18 * rng.standard_normal((batch.T, 8, 64)), dtype)
    y, lse = _run(q, cache, x, batch, dtype=torch.float32)   # (fp16 ends at 65504, these do not)
    wy, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 0.125)
    _within(_np(y), wy, R.rounded(wy, e, "float32"), "y")
    _within(_np(lse), wl, le, "lse")
    for _ in range(50):
        again = _run(q, cache, x, batch, dtype=torch.float32)
        assert torch.equal(again[0], y) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kernel", ["tc", "tc fp16"])
def test_first_tiles_come_to_where_the_shares_were_found(cuda_lib, kernel):
    """Many sequences of one tile: the first codes of a block arrive where its prefix sums were just read.  Against 64
    bits, and the same bits again and again."""
    import torch
    q = cuda_lib
    dtype, new, _ = KERNELS[kernel]
    rng = np.random.default_rng(71)
    batch = R.Batch(rng, [new] * 40, rng.integers(new, 129, 40).tolist(), 16)
    cache, codes, scales = _cache(q, rng, batch, 2, 64, spread=20)
    x, xv = _as(2.0 ** -18 * rng.standard_normal((batch.T, 8, 64)), dtype)
    y, lse = _run(q, cache, x, batch, dtype=torch.float32)   # (fp16 ends at 65504, these do not)
    wy, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 0.125)
    _within(_np(y), wy, R.rounded(wy, e, "float32"), "y")
    _within(_np(lse), wl, le, "lse")
    for _ in range(50):
        again = _run(q, cache, x, batch, dtype=torch.float32)
        assert torch.equal(again[0], y) and torch.equal(again[1], lse)


# ---------------------------------------------------------------------------
# The formula in 64 bits and the bounds that the header gives
# ---------------------------------------------------------------------------
U = {"float32": 2.0 ** -20, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -11}
QUERY = {"float32": 2.0 ** -38, "float16": 2.0 ** -21, "bfloat16": 2.0 ** -21}  # of the head's largest value


def _exact(x, dtype, codes, scales, batch, scale, causal=True, window=0, small=False):
    """(y, lse, bound of y before its rounding, bound of lse).  small: some query values are far below the head's largest,
    so that what they may be off counts: a score then by d = |scale| max(QUERY m, 2^-114) sum |k_ji| at most, and a
    probability by exp(2 d) - 1 of itself.  A NaN code of a value: NaN in that element of the rows that see it."""
    T, Hq, D = x.shape
    H = codes[0].shape[1]
    x = x.astype(np.float64)
    y, ey, lse, el = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b, (m, n) in enumerate(zip(batch.new, batch.lengths)):
        if n == 0 or m == 0:
            continue
        ids = batch.table[b, :-(-n // batch.page)]
        flat = lambda a: a.transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
        K, V = (flat(R.VALUES[codes[i][ids]] * scales[i][ids].astype(np.float64)[:, :, None, None]) for i in range(2))
        s = np.repeat(scales[1][ids].astype(np.float64), batch.page, 0)[:n]
        nan, V = np.isnan(V), np.nan_to_num(V)
        pos, j = np.arange(n - m, n)[:, None], np.arange(n)[None, :]
        seen = (j <= pos) & ((j > pos - window) if window else True) if causal else np.ones((m, n), bool)
        rows, some, count = slice(batch.offsets[b], batch.offsets[b + 1]), seen.any(axis=1), seen.sum(axis=1)
        for h in range(Hq):
            g, Q = h // (Hq // H), x[rows, h]
            z = np.where(seen, scale * (Q @ K[g].T), -np.inf)
            X = np.where(seen, abs(scale) * (np.abs(Q) @ np.abs(K[g]).T), 0).max(axis=1)
            top = np.where(some, z.max(axis=1), 0)
            p = np.exp(z - top[:, None])
            total = np.where(some, p.sum(axis=1), 1)
            p /= total[:, None]
            c = (count + (D + 64) * (1 + X)) * 2.0 ** -22
            if small:
                off = np.maximum(QUERY[dtype] * np.abs(Q).max(axis=1), 2.0 ** -114)
                c = c + np.expm1(2 * abs(scale) * off * np.where(seen, np.abs(K[g]).sum(axis=1), 0).max(axis=1))
            y[rows, h] = np.where((seen.astype(np.float64) @ nan[g]) > 0, np.nan, p @ V[g])
            ey[rows, h] = (U[dtype] + c)[:, None] * (p @ np.abs(V[g])) + (count * 2.0 ** -22 * (p * s[:, g]).max(axis=1))[:, None]
            lse[rows, h] = np.where(some, top + np.log(total), -np.inf)
            el[rows, h] = c + 2.0 ** -22 * np.where(some, np.abs(lse[rows, h]), 0)
    return y, lse, ey, el


def _against(q, cache, codes, scales, batch, x, xv, dtype, scale=0.125, small=False, **k):
    """The call with fp32 results against _exact."""
    import torch
    got = _run(q, cache, x, batch, scale=scale, dtype=torch.float32, **k)
    wy, wl, ey, el = _exact(xv, dtype, codes, scales, batch, scale, small=small, **k)
    _within(_np(got[0]), wy, R.rounded(wy, ey, "float32"), "y")
    _within(_np(got[1]), wl, el, "lse")
    return got


def _put(cache, codes, scales):
    import torch
    for t, a in zip((cache.k, cache.v), codes):
        t.view(torch.uint8).copy_(_t(a))
    for t, a in zip((cache.k_scale, cache.v_scale), scales):
        t.copy_(_t(a.astype(np.float32)))


@pytest.mark.parametrize("kernel", KERNELS)
def test_windows_near_the_end_of_32_bits(cuda_lib, kernel):
    """A window of 2^31 - 1 is none, also where a sequence has more rows than tokens."""
    import torch
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    new = max(new, 8)
    rng = np.random.default_rng(72)
    for n, lengths in (([new] * 6, [new - 3] * 6), ([new] * 6, [new - 3, new + 200, 0, 1, new, 300])):
        batch = R.Batch(rng, n, lengths, 16, width=width)
        cache, codes, scales = _cache(q, rng, batch, 2, 64)
        x, xv = _as(rng.standard_normal((batch.T, 8, 64)), dtype)
        none = _against(q, cache, codes, scales, batch, x, xv, dtype)
        for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 4):
            got = _against(q, cache, codes, scales, batch, x, xv, dtype, window=window)
            assert torch.equal(got[0], none[0]) and torch.equal(got[1], none[1])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_many_rows_of_few_tokens_and_a_window_as_wide_as_the_table(cuda_lib, dtype):
    """1300 rows of 5 tokens, a table for 2^31 - 1024 tokens, a window of 2^31 - 1200."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(73)
    small = R.Batch(rng, [1300], [5], 128)
    cache, codes, scales = _cache(q, rng, small, 1, 64)
    x, xv = _as(rng.standard_normal((1300, 1, 64)), dtype)
    wide = torch.zeros(1, (1 << 24) - 8, dtype=torch.int32, device="cuda")
    wide[0, 0] = int(small.table[0, 0])
    y, lse = q.qmm_kv_attention(cache, x, wide, _i32([5]), offsets=_i32([0, 1300]), window=2 ** 31 - 1200, dtype=torch.float32, lse=True)
    assert q.qmm_device_status() == 0
    wy, wl, ey, el = _exact(xv, dtype, codes, scales, small, 0.125)
    _within(_np(y), wy, R.rounded(wy, ey, "float32"), "y")
    _within(_np(lse), wl, el, "lse")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("low,high", [(-100, 28), (-100, 40), (-100, 100), (-60, 100), (-100, -5)])
def test_pages_of_value_scales_far_apart(cuda_lib, kernel, low, high):
    """Pages of zeros, whose scale is 2^-100, or of tiny values beside pages of large ones: they have their share in the
    sum of the probabilities, whichever come first and wherever a sequence is cut."""
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    rng = np.random.default_rng(74)
    for page, lengths, first in ((16, [900, 300, 77], None), (64, [9000, 200, 3000], low), (64, [9000, 200, 3000], high)):
        batch = R.Batch(rng, [new] * 3, [max(n, new) for n in lengths], page, width=2 * width)
        cache, codes, scales = _cache(q, rng, batch, 2, 64)
        for b in range(3):
            ids = batch.table[b, :-(-batch.lengths[b] // page)]
            if first is None:
                tiny = rng.integers(0, 2, (len(ids), 2)) > 0
            else:
                tiny = np.repeat((np.arange(len(ids)) < len(ids) // 2)[:, None] == (first == low), 2, 1)
            scales[1][ids] = np.where(tiny, 2.0 ** low, 2.0 ** high)
            if low == -100:
                codes[1][ids] = np.where(tiny[:, :, None, None], 0, codes[1][ids])
        _put(cache, codes, scales)
        x, xv = _as(0.1 * rng.standard_normal((batch.T, 8, 64)), dtype)
        _against(q, cache, codes, scales, batch, x, xv, dtype)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("window", [0, 60])
def test_a_nan_code_of_a_value_reaches_its_element_alone(cuda_lib, kernel, window):
    """Of the rows that see the token, in tiles that all rows see and in tiles that a mask cuts; the other elements and
    the log of the sum are as if the value was none.  (Codes of -0 beside it are no NaN.)"""
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    rng = np.random.default_rng(75)
    for dim, longest in ((64, 300), (48, 300), (128, 300), (256, 300), (128, 5003)):
        batch = R.Batch(rng, [new] * 3, [max(n, new) for n in (longest, 140, 129)], 64, width=2 * width + longest // 64)
        cache, codes, scales = _cache(q, rng, batch, 2, dim)
        for b in range(3):
            n = batch.lengths[b]
            for j in {3, 126, n // 2, n - new, n - 1 - new // 2, n - 1, max(0, n - 60), max(0, n - 61)}:
                at = codes[1][batch.table[b, j // 64], j % 2, j % 64]
                at[rng.integers(0, dim, 7)] = 0x80
                at[rng.integers(0, dim, 2)] = rng.choice([0x7f, 0xff], 2)
            codes[1][batch.table[b, (n - 1) // 64], :, (n - 1) % 64 + 1:] = 0x7f   # behind the end
        _put(cache, codes, scales)
        x, xv = _as(rng.standard_normal((batch.T, 8, dim)), dtype)
        y, _ = _against(q, cache, codes, scales, batch, x, xv, dtype, window=window)
        nan = np.isnan(_np(y))
        assert nan.any() and not nan.all(axis=2).any()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("scale,large", [(0.0, 100), (1e-33, 100), (-1e-33, 100), (1e-36, 110)])
def test_scales_of_the_scores_that_nearly_vanish(cuda_lib, kernel, scale, large):
    """With 0 every row is the mean of what it sees, whatever the keys are; tiny scales of large keys."""
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    rng = np.random.default_rng(76)
    batch = R.Batch(rng, [new] * 3, [max(n, new) for n in (300, 140, 129)], 64, width=2 * width)
    cache, codes, scales = _cache(q, rng, batch, 2, 64)
    scales[0] = np.full_like(scales[0], 2.0 ** large)
    _put(cache, codes, scales)
    x, xv = _as(rng.standard_normal((batch.T, 8, 64)), dtype)
    _against(q, cache, codes, scales, batch, x, xv, dtype, scale=scale)


# ---------------------------------------------------------------------------
# offsets that fall
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("offsets", [[0, 100, 50, 200], [0, 10, 1000000, 150, 200], [0, 60, -5000, 130, 200], [0, 100, 99, 200]])
@pytest.mark.parametrize("what", ["append", "bfloat16", "float32", "few"])
def test_offsets_that_fall_are_always_reported(cuda_lib, what, offsets):
    """Wherever they lie between others; rows behind the last sequence and what the batch does not hold stay."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(79)
    B, T = len(offsets) - 1, 200
    if what == "few":
        offsets = [min(o, 10 ** 6) // 25 for o in offsets]
        T = 8
    cache = q.KvCache.empty(20 * B, 2, page=16, dim=64)
    table, lengths = _i32(np.arange(20 * B).reshape(B, 20)), _i32([250] * B)
    dtype = torch.float32 if what == "float32" else torch.bfloat16
    x = torch.randn(T + 4, 8, 64, device="cuda", dtype=dtype)
    y = torch.full_like(x, 7.0)
    if what == "append":
        q.qmm_kv_append(cache, x[:, :2], x[:, :2], table, lengths, offsets=_i32(offsets))
    else:
        q.qmm_kv_attention(cache, x, table, lengths, offsets=_i32(offsets), y=y)
    assert q.qmm_device_status() == q.QMM_EINDEX and q.qmm_device_status() == 0
    assert bool((y[T:] == 7).all())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("lengths,window", [([32769], 0), ([20001, 77, 9000], 0), ([20001, 300, 9000], 5000),
                                            ([3000 + 97 * b for b in range(40)], 0)])
def test_no_tile_of_a_long_sequence_is_lost_or_counted_twice(cuda_lib, kernel, lengths, window):
    """Queries of zero, so that every token counts the same, and values of 1 in one element for each 128 tokens: the
    results are the numbers of tokens over their sum.  Both are whole numbers times a power of two, exact in fp32: a
    division, a product and an exponential of 0 are left, 2^-20 at most together, and a tile is 2^-8 or more of a sum."""
    import torch
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    rng = np.random.default_rng(76)
    dim, heads = 128, 2
    batch = R.Batch(rng, [new] * len(lengths), lengths, 64, width=width)
    codes = rng.integers(0, 127, (batch.pages, heads, 64, dim), np.uint8)
    values = np.zeros((batch.pages, heads, 64, dim), np.uint8)
    for b, n in enumerate(lengths):
        for page in range(-(-n // 64)):
            values[batch.table[b, page], :, :, page // 2 % dim] = 0x38   # 1.0
    ones = torch.ones(batch.pages, heads, device="cuda")
    cache = q.KvCache(_t(codes).view(torch.float8_e4m3fn), _t(values).view(torch.float8_e4m3fn), ones, ones.clone())
    x, _ = _as(np.zeros((batch.T, 4 * heads, dim)), dtype)
    y, lse = _run(q, cache, x, batch, dtype=torch.float32, window=window)
    end = batch.positions() + 1
    begin = np.maximum(end - window, 0) if window else np.zeros_like(end)
    counts = np.zeros((batch.T, dim))
    for tile in range(-(-max(lengths) // 128)):
        counts[:, tile % dim] += np.clip(np.minimum(end, 128 * tile + 128) - np.maximum(begin, 128 * tile), 0, None)
    n = (end - begin).astype(np.float64)
    want = np.broadcast_to((counts / n[:, None])[:, None], y.shape)
    _within(_np(y), want, 2.0 ** -20 * want, "y")
    wl = np.broadcast_to(np.log(n)[:, None], lse.shape)
    _within(_np(lse), wl, 2.0 ** -20 * (1 + wl), "lse")


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_ramp_over_pairs_by_frequencies_of_ones_own(cuda_lib, interleaved):
    """What qmm_rope_table says of checkpoints tuned with a ramp over the pairs: frequencies and factor as given there."""
    q = cuda_lib
    rot, base, scale, original, low, high = 128, 10000.0, 16.0, 8192, 1.0, 32.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    ends = [rot / 2 * math.log(original / (2 * math.pi * r)) / math.log(base) for r in (high, low)]
    keep = 1.0 - np.clip((i - ends[0]) / (ends[1] - ends[0]), 0.0, 1.0)
    f = f * keep + f / scale * (1.0 - keep)
    factor = 0.1 * math.log(scale) + 1.0
    rng = np.random.default_rng(77)
    x, xv = _as(rng.standard_normal((60, 2, rot)), "float32")
    pos = rng.integers(0, 100000, 60).astype(np.int32)
    y = q.qmm_rope(x, q.qmm_rope_table(rot, freqs=f, factor=factor, interleaved=interleaved), _t(pos))
    want, e = R.rope(xv, pos, f, interleaved, False, factor)
    _within(_np(y), want, R.rounded(want, e, "float32"))

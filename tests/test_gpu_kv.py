"""The position rotation, the append to the paged 8-bit cache and the attention over it on the GPU, against 64 bits
(kv_reference.py): from one token to long sequences, odd and ragged sizes, every type, pitches, empty rows."""
import math

import numpy as np
import pytest

import kv_reference as R

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _as(a, dtype):
    """float32 numpy values -> (device tensor of dtype, the values it holds: float32 for float32, else float64)."""
    import torch
    t = _t(np.asarray(a, np.float32)).to(getattr(torch, dtype))
    v = t.float().cpu().numpy()
    return t, v if dtype == "float32" else v.astype(np.float64)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _u8(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def _within(got, want, bound, what=""):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= bound))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[:3].tolist()}, worst "
                           f"{np.nanmax(np.where(bad, np.abs(got - want) / np.maximum(bound, 1e-300), 0)):.3g} bounds")


def _table(q, rot, interleaved=False, **k):
    return q.qmm_rope_table(rot, interleaved=interleaved, **k)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,heads,dim,rot,interleaved,inverse", [
    (1, 1, 2, 2, False, False), (1, 32, 128, 128, False, False), (7, 3, 80, 40, False, True), (5, 5, 96, 48, True, False),
    (33, 1, 64, 62, True, True), (19, 2, 256, 256, False, False), (3, 7, 66, 6, False, False), (1000, 9, 128, 64, True, False),
    (2, 3, 64, 0, False, False), (700, 40, 128, 128, False, True)])
def test_rope(cuda_lib, dtype, T, heads, dim, rot, interleaved, inverse):
    q = cuda_lib
    rng = np.random.default_rng(T + dim)
    x, xv = _as(rng.standard_normal((T, heads, dim)), dtype)
    pos = rng.integers(-5, 200000, T).astype(np.int32)
    table = _table(q, rot, interleaved, base=500000.0, factor=1.25)
    y = q.qmm_rope(x, table, _t(pos), inverse=inverse)
    want, e = R.rope(xv, pos, R.frequencies(rot, 500000.0), interleaved, inverse, 1.25)
    assert y.dtype == x.dtype and y.shape == x.shape
    _within(_np(y), want, R.rounded(want, e, dtype))


def test_rope_far_positions(cuda_lib):
    """The largest and the smallest position: the angle is exact where pos * frequency in fp32 has no correct digit."""
    q = cuda_lib
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 123456789], np.int32)
    x, xv = _as(np.random.default_rng(0).standard_normal((len(pos), 2, 64)), "float32")
    y = q.qmm_rope(x, _table(q, 64), _t(pos))
    # the frequencies in 64 bits are 2^-53 off, the angle of position 2^31 6e-7: within the bound, 2^-21, but not far
    want, e = R.rope(xv, pos, R.frequencies(64))
    far = 2.0 ** 31 * 2.0 ** -52 * (np.abs(xv[..., :32]) + np.abs(xv[..., 32:]))
    _within(_np(y), want, R.rounded(want, e + np.concatenate([far, far], axis=2), "float32"))


@pytest.mark.parametrize("scaling,extra", [("linear", {}), ("ntk", {}), ("parts", {"original": 4096}),
                                           ("parts", {"original": 8192, "low": 2.0, "high": 20.0}), ("yarn", {"original": 4096})])
def test_rope_scalings(cuda_lib, scaling, extra):
    q = cuda_lib
    rng = np.random.default_rng(3)
    x, xv = _as(rng.standard_normal((50, 2, 96)), "float32")
    pos = rng.integers(0, 100000, 50).astype(np.int32)
    y = q.qmm_rope(x, _table(q, 96, scaling=scaling, scale=8.0, **extra), _t(pos))
    if scaling == "yarn":
        f, factor = R.frequencies(96, scaling="parts", scale=8.0, high=32.0, **extra), 0.1 * math.log(8.0) + 1
    else:
        f, factor = R.frequencies(96, scaling=scaling, scale=8.0, **extra), 1.0
    want, e = R.rope(xv, pos, f, factor=factor)
    _within(_np(y), want, R.rounded(want, e, "float32"))


def test_rope_own_frequencies(cuda_lib):
    q = cuda_lib
    f = np.array([7.5, 0.25, 0.0, 1e-6])   # (more than a full turn per position among them)
    x, xv = _as(np.random.default_rng(4).standard_normal((9, 1, 8)), "float32")
    pos = np.arange(9, dtype=np.int32) * 1001
    y = q.qmm_rope(x, q.qmm_rope_table(8, freqs=f), _t(pos))
    want, e = R.rope(xv, pos, f)
    _within(_np(y), want, R.rounded(want, e, "float32"))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(cuda_lib, interleaved):
    """Against differences: the rotation is linear, so <g, R(x + d) - R(x)> = <R^T g, d>."""
    q = cuda_lib
    rng = np.random.default_rng(5)
    pos = _t(rng.integers(0, 30000, 11).astype(np.int32))
    table = _table(q, 48, interleaved, factor=1.5)
    x, d, g = (_as(rng.standard_normal((11, 3, 64)), "float32")[0] for _ in range(3))
    moved = (q.qmm_rope(x + d, table, pos).double() - q.qmm_rope(x, table, pos).double())
    grad = q.qmm_rope(g, table, pos, inverse=True).double()
    left, right = (g.double() * moved).sum(), (grad * d.double()).sum()
    # each side's values are off by a few 2^-21 of what they are made of
    bound = 8 * 2.0 ** -21 * 1.5 * float((g.double().abs().sum() * (x.abs() + d.abs()).double().max()))
    assert abs(float(left - right)) <= bound
    assert float((grad * d.double()).abs().sum()) > 100 * bound


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_rope_pitches_and_in_place(cuda_lib, dtype):
    """Heads of a fused projection, heads before rows, an odd start; the result in place and into pitched rows."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(6)
    pos = rng.integers(0, 5000, 6).astype(np.int32)
    table, f = _table(q, 64), R.frequencies(64)
    for view in (lambda b: b[:6 * 7 * 80].view(6, 7, 80)[:, 2:6, :64], lambda b: b[:4 * 6 * 64].view(4, 6, 64).transpose(0, 1),
                 lambda b: b[1:1 + 6 * 4 * 65].view(6, 4, 65)[:, :, :64]):
        buf = _as(rng.standard_normal(4000), dtype)[0]
        x = view(buf)
        xv = x.float().cpu().numpy()
        want, e = R.rope(xv, pos, f)
        b = R.rounded(want, e, dtype)
        _within(_np(q.qmm_rope(x, table, _t(pos))), want, b)
        before = buf.clone()
        out = torch.zeros_like(buf)
        q.qmm_rope(x, table, _t(pos), y=view(out))
        _within(_np(view(out)), want, b)
        view(out).zero_()
        assert not out.any()                         # nothing between the rows was written
        assert torch.equal(buf, before)
        assert q.qmm_rope(x, table, _t(pos), y=x) is x
        _within(_np(x), want, b)
        x.copy_(view(before))
        assert torch.equal(buf, before)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _cache(q, rng, batch, heads, dim, spread=3, wide=None):
    """A cache of random pages; scales 2^-spread .. 2^spread of what unit values need."""
    import torch
    n = batch.pages
    codes = [R.codes_of(rng.standard_normal((n, heads, batch.page, dim)) * 112) for _ in range(2)]
    scales = [(2.0 ** rng.integers(-spread, spread + 1, (n, heads)) / 128).astype(np.float32) for _ in range(2)]
    t = [_t(c).view(torch.float8_e4m3fn) for c in codes] + [_t(s) for s in scales]
    return q.KvCache(*t), codes, scales


def _check_append(q, cache, codes, scales, batch, kv, ke, vv):
    """The cache against the reference: values bit for bit; keys, which were turned, within a rounding of them."""
    vc, vs = R.append(codes[1], scales[1], np.asarray(vv, np.float64), batch)
    assert np.array_equal(cache.v_scale.cpu().numpy(), vs)
    assert np.array_equal(_u8(cache.v), vc)
    kc, ks = R.append(codes[0], scales[0], kv, batch)
    assert np.array_equal(cache.k_scale.cpu().numpy(), ks)      # (no maximum is near a power of two here)
    got, want = _u8(cache.k), kc
    new = np.zeros(got.shape, bool)
    exact, err = np.zeros(got.shape), np.zeros(got.shape)
    pos, r = batch.positions(), 0
    for b, m in enumerate(batch.new):
        for _ in range(m):
            p, slot = batch.table[b, pos[r] // batch.page], pos[r] % batch.page
            new[p, :, slot], exact[p, :, slot], err[p, :, slot] = True, kv[r], ke[r]
            r += 1
    assert np.array_equal(got[~new], want[~new])
    s = ks[:, :, None, None]
    # half a step of e4m3 around the value, and what the rotation may be off
    half = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * s)
    _within((R.VALUES[got] * s)[new], exact[new], (half + 2 * err)[new], "keys")
    assert (got != want).mean() < 1e-3


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,heads,dim,rot,interleaved,new,lengths", [
    (64, 8, 128, 128, False, [1] * 5, [1, 64, 65, 300, 128]),       # single tokens: first, last and middle slots of a page
    (16, 1, 16, 16, True, [1], [1]),
    (16, 2, 80, 40, False, [1, 1, 1], [33, 16, 2]),
    (32, 3, 96, 48, True, [5, 70, 0, 31], [5, 99, 7, 64]),           # a sequence without new rows
    (128, 2, 256, 256, False, [129, 3], [300, 3]),
    (128, 3, 128, 128, False, [200, 256], [200, 700]),
    (64, 2, 64, 0, False, [67, 1], [131, 65]),
    (64, 2, 64, 62, False, [67, 1], [131, 65])])                    # (no runs of four pairs)
def test_append(cuda_lib, dtype, page, heads, dim, rot, interleaved, new, lengths):
    q = cuda_lib
    rng = np.random.default_rng(dim + len(new))
    batch = R.Batch(rng, new, lengths, page)
    cache, codes, scales = _cache(q, rng, batch, heads, dim)
    rows = lambda h: (rng.standard_normal((batch.T, h, dim)) * 2.0 ** rng.integers(-3, 4, (batch.T, h, 1))).astype(np.float32)
    (k, kv), (v, vv), (x, xv) = _as(rows(heads), dtype), _as(rows(heads), dtype), _as(rows(heads * 3), dtype)
    table = _table(q, rot, interleaved)
    single = all(n == 1 for n in new)
    got = q.qmm_kv_append(cache, k, v, _t(batch.table), _t(np.array(lengths, np.int32)),
                          offsets=None if single else _t(batch.offsets), rope=table, q=x)
    assert q.qmm_device_status() == 0
    f, pos = R.frequencies(rot), batch.positions()
    want, e = R.rope(xv, pos, f, interleaved)
    _within(_np(got), want, R.rounded(want, e, dtype), "queries")
    _check_append(q, cache, codes, scales, batch, *R.rope(kv, pos, f, interleaved), vv)


def test_append_without_rotation_or_with_other_positions(cuda_lib):
    q = cuda_lib
    rng = np.random.default_rng(7)
    batch = R.Batch(rng, [3, 40], [20, 41], 32)
    lengths, offsets, table = _t(np.array(batch.lengths, np.int32)), _t(batch.offsets), _t(batch.table)
    for positions in (None, rng.integers(0, 100000, batch.T).astype(np.int32)):
        cache, codes, scales = _cache(q, rng, batch, 2, 64)
        (k, kv), (v, vv) = (_as(rng.standard_normal((batch.T, 2, 64)), "bfloat16") for _ in range(2))
        if positions is None:
            assert q.qmm_kv_append(cache, k, v, table, lengths, offsets=offsets) is None
            _check_append(q, cache, codes, scales, batch, kv, np.zeros_like(kv), vv)
        else:
            q.qmm_kv_append(cache, k, v, table, lengths, offsets=offsets, rope=_table(q, 64), positions=_t(positions))
            _check_append(q, cache, codes, scales, batch, *R.rope(kv, positions, R.frequencies(64)), vv)


def test_append_token_by_token(cuda_lib):
    """A page filled one by one with growing and falling values, as decoding does: scales grow, what is held is rounded
    anew, and the page after it starts afresh."""
    q = cuda_lib
    rng = np.random.default_rng(8)
    cache = q.KvCache.empty(3, 1, page=16, dim=32)
    codes, scales = [_u8(cache.k), _u8(cache.v)], [cache.k_scale.cpu().numpy(), cache.v_scale.cpu().numpy()]
    table = np.array([[2, 0]], np.int32)
    for n in range(1, 23):
        x = (rng.standard_normal((1, 1, 32)) * 2.0 ** (7 * math.sin(n))).astype(np.float32)
        if n == 5:
            x[0, 0] = 0.0
        batch = R.Batch(rng, [1], [n], 16)
        batch.table = table
        q.qmm_kv_append(cache, _t(x), _t(-x), _t(table), _t(np.array([n], np.int32)))
        codes[0], scales[0] = R.append(codes[0], scales[0], x.astype(np.float64), batch)
        codes[1], scales[1] = R.append(codes[1], scales[1], -x.astype(np.float64), batch)
        assert np.array_equal(_u8(cache.k), codes[0]) and np.array_equal(cache.k_scale.cpu().numpy(), scales[0])
        assert np.array_equal(_u8(cache.v), codes[1]) and np.array_equal(cache.v_scale.cpu().numpy(), scales[1])


def test_append_extremes(cuda_lib):
    """Zeros, subnormals, the largest floats, values on the border of a scale; a NaN or an infinity is a NaN code and
    changes neither the scale nor what lies beside it."""
    q = cuda_lib
    rng = np.random.default_rng(9)
    T = 12
    x = rng.standard_normal((T, 1, 16)).astype(np.float32)
    x[0] = 0.0
    x[1] = 1e-41
    x[2] *= 3e38 / np.abs(x[2]).max()
    x[3] *= 448.0 / np.abs(x[3]).max()
    x[3, 0, 5] = 448.0                       # scale 1
    x[4, 0, :] = 0.5
    x[4, 0, 5] = np.nextafter(np.float32(448.0), np.float32(1e9))   # scale 2
    x[5, 0, 3] = np.nan
    x[6, 0, 3], x[6, 0, 4] = np.inf, -np.inf
    x[7] = np.nan
    x[8] = 2.0 ** -99
    batch = R.Batch(rng, [1] * T, [1] * T, 16)
    cache, codes, scales = _cache(q, rng, batch, 1, 16)
    q.qmm_kv_append(cache, _t(x), _t(x), _t(batch.table), _t(np.ones(T, np.int32)))
    for i, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        want, ws = R.append(codes[i], scales[i], x.astype(np.float64), batch)
        assert np.array_equal(s.cpu().numpy(), ws)
        g = _u8(c)
        assert np.array_equal(np.where(g & 127 == 127, 127, g), np.where(want & 127 == 127, 127, want))


def test_append_pitches_and_queries_in_place(cuda_lib):
    """Queries, keys and values as parts of one projection; the turned queries in their place; rows behind the last
    sequence and everything between stay as they were."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(10)
    for dtype, pad in (("bfloat16", 0), ("float16", 1), ("float32", 0)):
        batch = R.Batch(rng, [4, 33], [30, 90], 64)
        T, Hq, H, D = batch.T + 5, 6, 2, 64
        buf = _as(rng.standard_normal((T, (Hq + 2 * H) * D + pad)), dtype)[0]
        x = buf[:, :(Hq + 2 * H) * D].unflatten(1, (Hq + 2 * H, D))
        h = x.float().cpu().numpy()[:batch.T].astype(np.float64)
        before = buf.clone()
        cache, codes, scales = _cache(q, rng, batch, H, D)
        got = q.qmm_kv_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], _t(batch.table), _t(np.array(batch.lengths, np.int32)),
                              offsets=_t(batch.offsets), rope=_table(q, D), q=x[:, :Hq], q_out=x[:, :Hq])
        f, pos = R.frequencies(D), batch.positions()
        want, e = R.rope(h[:, :Hq], pos, f)
        _within(_np(got)[:batch.T], want, R.rounded(want, e, dtype))
        _check_append(q, cache, codes, scales, batch, *R.rope(h[:, Hq:Hq + H], pos, f), h[:, Hq + H:])
        buf[:batch.T, :Hq * D] = before[:batch.T, :Hq * D]
        assert torch.equal(buf, before)


def test_append_refused_on_the_device(cuda_lib):
    """Lengths, offsets and pages out of range: skipped and reported, the other sequences and every other page as they
    should be."""
    q = cuda_lib
    rng = np.random.default_rng(11)
    new, lengths = [2, 3, 2, 2], [40, 35, 20, 20]
    for what in ("page", "negative page", "length", "short", "offset"):
        batch = R.Batch(rng, new, lengths, 16)
        cache, codes, scales = _cache(q, rng, batch, 2, 32)
        k, kv = _as(rng.standard_normal((batch.T, 2, 32)), "float32")
        table, lens, off = batch.table.copy(), np.array(lengths, np.int32), batch.offsets.copy()
        bad = 1
        if what == "page":
            table[1, 2] = batch.pages        # (tokens 32 to 34 are new)
        elif what == "negative page":
            table[1, 2] = -1
        elif what == "length":
            lens[1] = batch.table.shape[1] * 16 + 1
        elif what == "short":
            lens[1] = 2
        else:
            off[4], bad = batch.T + 1, 3
        q.qmm_kv_append(cache, k, k, _t(table), _t(lens), offsets=_t(off))
        assert q.qmm_device_status() == q.QMM_EINDEX and q.qmm_device_status() == 0
        good = R.Batch(rng, new, lengths, 16)
        good.table, good.new = batch.table, [0 if b == bad else n for b, n in enumerate(new)]
        want, ws = R.append(codes[0], scales[0], kv.astype(np.float64), good)
        assert np.array_equal(_u8(cache.k), want) and np.array_equal(cache.k_scale.cpu().numpy(), ws)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attend(q, rng, new, lengths, page, heads, group, dim, dtype, out=None, causal=True, window=0, scale=None, spread=3,
            single=None, qscale=1.0, width=0):
    import torch
    batch = R.Batch(rng, new, lengths, page, width=width)
    cache, codes, scales = _cache(q, rng, batch, heads, dim, spread)
    x, xv = _as(qscale * rng.standard_normal((batch.T, heads * group, dim)), dtype)
    single = all(n == 1 for n in new) if single is None else single
    y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _t(np.array(lengths, np.int32)),
                                offsets=None if single else _t(batch.offsets), scale=scale, causal=causal, window=window,
                                dtype=getattr(torch, out) if out else None, lse=True)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    want, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch,
                                  1 / math.sqrt(dim) if scale is None else scale, causal, window)
    out = out or dtype
    assert str(y.dtype) == "torch." + out
    bound = R.rounded(want, e, out)
    if out == "float16":                # whose largest value is 65504: from 65520 on a value rounds to infinity
        over = np.abs(want) - e >= 65520
        assert np.array_equal(_np(y)[over], np.copysign(np.inf, want[over]))
        want = np.where(np.abs(want) + e >= 65520, _np(y), want)
    _within(_np(y), want, bound, "y")
    _within(_np(lse), wl, le, "lse")
    return y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,heads,group,dim,lengths", [
    (64, 2, 4, 128, [1]), (64, 2, 4, 128, [0, 1, 127, 128, 129, 700]), (16, 3, 1, 64, [5, 16, 17, 1000]),
    (128, 1, 8, 256, [300, 4000]), (32, 2, 5, 80, [33, 257]), (16, 1, 3, 16, [1, 40]), (64, 1, 16, 96, [513, 64]),
    (64, 2, 33, 64, [200, 3]), (64, 8, 4, 128, [9001])])
def test_decode(cuda_lib, dtype, page, heads, group, dim, lengths):
    _attend(cuda_lib, np.random.default_rng(dim + len(lengths)), [1] * len(lengths), lengths, page, heads, group, dim, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,heads,group,dim,new,lengths,window", [
    (64, 2, 4, 128, [5, 1, 0, 3], [300, 65, 40, 3], 0),
    (16, 1, 2, 64, [17, 40], [17, 300], 0),
    (32, 2, 3, 80, [70], [70], 0),
    (128, 1, 8, 128, [130, 1, 257], [130, 900, 1200], 0),
    (16, 1, 1, 256, [40, 2], [90, 2], 7),                        # a window that ends inside a page
    (64, 2, 2, 64, [300, 200], [300, 777], 128),
    (64, 1, 4, 128, [200], [200], 1),                            # a row sees itself alone
    (64, 1, 4, 128, [9, 5], [4, 2], 0),                          # more rows than tokens: the first see nothing
    (64, 1, 6, 96, [64, 64, 64], [64, 128, 192], 1000)])
def test_rows(cuda_lib, dtype, page, heads, group, dim, new, lengths, window):
    _attend(cuda_lib, np.random.default_rng(dim + len(new)), new, lengths, page, heads, group, dim, dtype, window=window)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("page,heads,group,dim,new,lengths,window", [
    (64, 2, 4, 128, [3, 4, 0, 3], [3000, 650, 40, 3], 0), (64, 2, 4, 128, [5, 8], [5000, 129], 0), (32, 3, 5, 80, [2, 3], [700, 5], 0),
    (16, 2, 8, 64, [4, 4, 4], [90, 1000, 4], 0), (128, 1, 13, 96, [1, 1], [2000, 1], 0), (16, 2, 2, 48, [8, 8], [900, 30], 77),
    (64, 1, 4, 16, [7, 5], [4, 2], 0), (64, 2, 1, 128, [30, 20], [300, 200], 1), (64, 2, 16, 112, [1, 1, 1], [0, 400, 16], 0)])
def test_few_rows_of_sequences_that_may_be_long(cuda_lib, dtype, page, heads, group, dim, new, lengths, window):
    """9 to 32 rows per cache head, tables of many pages."""
    width = -(-8 * 160 * 128 // (len(new) * heads * page)) + 1
    for scale, qscale in ((None, 1.0), (-0.2, 3.0)):
        _attend(cuda_lib, np.random.default_rng(dim + len(new)), new, lengths, page, heads, group, dim, dtype, window=window,
                width=width, scale=scale, qscale=qscale)
    if not window:
        _attend(cuda_lib, np.random.default_rng(3), new, lengths, page, heads, group, dim, dtype, causal=False, width=width, spread=20)


@pytest.mark.parametrize("dtype,out", [("float32", "bfloat16"), ("bfloat16", "float32"), ("float16", "bfloat16")])
def test_attention_result_types_scale_and_all_tokens(cuda_lib, dtype, out):
    rng = np.random.default_rng(1)
    _attend(cuda_lib, rng, [3, 50], [200, 130], 64, 2, 4, 128, dtype, out=out, causal=False, scale=0.3)
    _attend(cuda_lib, rng, [1, 1], [200, 130], 64, 2, 4, 64, dtype, out=out, causal=False, scale=-0.05)
    _attend(cuda_lib, rng, [200], [260], 64, 2, 4, 128, dtype, out=out, causal=False)
    _attend(cuda_lib, rng, [5], [2], 64, 2, 4, 128, dtype, out=out, causal=False)
    _attend(cuda_lib, rng, [5, 3], [0, 0], 64, 2, 4, 128, dtype, out=out, causal=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 40])
def test_attention_with_scales_far_apart(cuda_lib, dtype, new):
    """Pages whose scales differ by 2^60, sharp and flat rows."""
    rng = np.random.default_rng(2)
    _attend(cuda_lib, rng, [new, new], [400, 77], 16, 2, 4, 64, dtype, spread=30, qscale=2.0 ** -28)
    _attend(cuda_lib, rng, [new, new], [400, 77], 16, 2, 4, 64, dtype, qscale=50.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,width,large", [(1, 0, 112), (4, 700, 112), (70, 0, 112), (1, 0, -100), (4, 700, -100), (70, 0, -100)])
def test_value_scales_at_the_ends_of_their_range(cuda_lib, dtype, new, width, large):
    """Value scales of 2^112 and 2^-100, where sums of probabilities over them come near the ends of fp32."""
    q = cuda_lib
    rng = np.random.default_rng(63)
    batch = R.Batch(rng, [new, new], [900, 300], 64, width=width)
    cache, codes, scales = _cache(q, rng, batch, 2, 64)
    scales[1][:] = 2.0 ** large
    cache.v_scale.copy_(_t(scales[1]))
    x, xv = _as(rng.standard_normal((batch.T, 8, 64)), dtype)
    y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _t(np.array(batch.lengths, np.int32)), offsets=_t(batch.offsets),
                                dtype=__import__("torch").float32, lse=True)
    assert q.qmm_device_status() == 0
    wy, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 0.125)
    _within(_np(y), wy, R.rounded(wy, e, "float32"), "y")
    _within(_np(lse), wl, le, "lse")


def test_nan_in_the_values_of_a_masked_token(cuda_lib):
    """A NaN among the values of a token makes the rows that see it NaN and no other, whatever tile they share; behind
    the end of a sequence, on a page that only other sequences know and outside the window it reaches nobody."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(12)
    for dtype, new, window, width in (("float32", 40, 0, 0), ("bfloat16", 3, 0, 0), ("bfloat16", 200, 0, 0), ("float16", 200, 50, 0),
                                      ("bfloat16", 200, 50, 0), ("bfloat16", 10, 0, 700), ("float16", 6, 0, 700), ("float32", 10, 0, 700)):
        batch = R.Batch(rng, [new, new], [300, 260], 64, width=width)
        cache, codes, scales = _cache(q, rng, batch, 2, 64)
        x = _as(rng.standard_normal((batch.T, 4, 64)), dtype)[0]
        args = (x, _t(batch.table), _t(np.array(batch.lengths, np.int32)), _t(batch.offsets))
        run = lambda c: _np(q.qmm_kv_attention(c, args[0], args[1], args[2], offsets=args[3], window=window))
        want = run(cache)
        v = cache.v.view(torch.uint8)
        k = cache.k.view(torch.uint8)
        spots = [298, 299] if new < 100 else [150, 297]     # tokens of the first sequence, of the second none
        for j in spots:
            v[int(batch.table[0, j // 64]), 1, j % 64, 5] = 127 if j % 2 else 255
        for c in (k, v):                                    # behind the ends, and pages of nobody
            c[int(batch.table[0, 4]), :, 300 - 256:] = 127
            c[int(batch.table[1, 4]), :, 260 - 256:] = 255
            c[[p for p in range(batch.pages) if p not in set(batch.table[batch.table >= 0].tolist())]] = 127
        got = run(cache)
        pos = np.arange(300 - new, 300)
        sees = np.zeros(batch.T, bool)
        for j in spots:
            sees[:new] |= (pos >= j) & ((pos < j + window) if window else True)
        assert sees.any() and not sees[:new].all()
        poisoned = np.zeros(got.shape, bool)
        poisoned[sees, 2:] = True                           # the query heads of cache head 1
        assert np.array_equal(got[~poisoned], want[~poisoned])
        assert np.isnan(got[poisoned].reshape(-1, 64)[:, 5]).all()
        assert q.qmm_device_status() == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("new", [1, 200])
def test_one_large_query_value_leaves_the_others_theirs(cuda_lib, dtype, new):
    """A channel with queries 2^12 times the others' and keys of 0: no share in any score, and the others keep their bits
    but for those that are smaller still."""
    q = cuda_lib
    rng = np.random.default_rng(61)
    H, D = 2, 64
    batch = R.Batch(rng, [new], [500], 64)
    cache, codes, scales = _cache(q, rng, batch, H, D)
    codes[0][..., 5] = 0
    cache.k.view(__import__("torch").uint8).copy_(_t(codes[0]))
    values = rng.standard_normal((batch.T, 4, D))
    values[..., 5] = 4096.0 * np.where(values[..., 5] < 0, -1, 1)
    x, xv = _as(values, dtype)
    y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _t(np.array([500], np.int32)), offsets=_t(batch.offsets), lse=True)
    wy, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, D ** -0.5, small=True)
    _within(_np(y), wy, R.rounded(wy, e, dtype), "y")
    _within(_np(lse), wl, le, "lse")
    assert q.qmm_device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,width", [(1, 0), (200, 0), (6, 700)])
def test_nan_and_infinities_in_queries_and_keys(cuda_lib, dtype, new, width):
    """In a head's query: its results are NaN (also where every score is -inf).  In a key: those of the rows that see the
    token.  All others are as they should be."""
    q = cuda_lib
    rng = np.random.default_rng(62)
    H, D, lengths = 2, 64, [500, 300]
    batch = R.Batch(rng, [new, new], lengths, 64, width=width)
    cache, codes, scales = _cache(q, rng, batch, H, D)
    codes[0][..., 7] = 0x38                       # 1, so that one infinite query value decides all scores
    at = 300 - new // 2 - 1                       # of the second sequence: seen by half of its rows (by its only one)
    codes[0][batch.table[1, at // 64], 1, at % 64, 9] = 0x7f
    cache.k.view(__import__("torch").uint8).copy_(_t(codes[0]))
    values = rng.standard_normal((batch.T, 4, D))
    bad = np.zeros((batch.T, 4), bool)
    for row, head, i, v in ((0, 1, 3, np.nan), (0, 2, 7, np.inf), (0, 3, 7, -np.inf), (batch.T - 1, 0, 0, np.nan), (new // 3, 0, 63, np.inf)):
        values[row, head, i] = v
        bad[row, head] = True
    if new == 1:
        bad[1, 2:] = True
    else:
        bad[batch.T - 1 - new // 2:, 2:] = True   # rows from position `at` on, heads of cache head 1
    x, xv = _as(values, dtype)
    y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _t(np.array(lengths, np.int32)), offsets=_t(batch.offsets), lse=True)
    assert q.qmm_device_status() == 0
    codes[0][codes[0] == 0x7f] = 0
    wy, wl, e, le = R.attention(np.where(np.isfinite(xv), xv, 0).astype(xv.dtype), codes[0], scales[0], codes[1], scales[1], batch, D ** -0.5)
    y, lse = _np(y), _np(lse)
    assert np.isnan(y[bad]).all() and np.isnan(lse[bad]).all()
    _within(y[~bad], wy[~bad], R.rounded(wy, e, dtype)[~bad], "y")
    _within(lse[~bad], wl[~bad], le[~bad], "lse")

"""The attention layer's calls as programs use them, on the GPU: prompt, chunks and single tokens one after another, in a
captured graph, on several streams and from several threads, on parts of larger tensors, after a wait that ran out."""
import math
import threading

import numpy as np
import pytest

import kv_reference as R
from test_gpu_kv import _as, _cache, _np, _t, _u8, _within

pytestmark = pytest.mark.gpu


def _i32(a):
    return _t(np.asarray(a, np.int32))


@pytest.mark.parametrize("dtype,page,interleaved", [("bfloat16", 16, False), ("float32", 32, True), ("float16", 64, False)])
def test_a_layer_over_a_conversation(cuda_lib, dtype, page, interleaved):
    """Two sequences: prompts, then chunks, then token by token; after each step the cache and the results against the
    reference, which goes through the same steps from the cache that it holds itself."""
    q = cuda_lib
    rng = np.random.default_rng(20)
    Hq, H, D = 6, 2, 64
    table = rng.permutation(64).astype(np.int32).reshape(2, 32)[:, :512 // page]
    cache = q.KvCache.empty(64, H, page=page, dim=D)
    rope, f = q.qmm_rope_table(D, interleaved=interleaved, scaling="parts", scale=4.0, original=256), \
        R.frequencies(D, scaling="parts", scale=4.0, original=256)
    have = [0, 0]
    for new in ((90, 33), (40, 41), (1, 1), (1, 1), (0, 7), (200, 1), (1, 1)):
        have = [a + b for a, b in zip(have, new)]
        batch = R.Batch(rng, new, have, page)
        batch.table = table
        T = batch.T
        (x, xv), (k, kv), (v, vv) = (_as(rng.standard_normal((T, n, D)), dtype) for n in (Hq, H, H))
        single = all(n == 1 for n in new)
        args = (_t(table), _i32(have))
        off = None if single else _t(batch.offsets)
        before = [_u8(cache.k), cache.k_scale.cpu().numpy(), _u8(cache.v), cache.v_scale.cpu().numpy()]
        turned = q.qmm_kv_append(cache, k, v, *args, offsets=off, rope=rope, q=x)
        y, lse = q.qmm_kv_attention(cache, turned, *args, offsets=off, lse=True)
        assert q.qmm_device_status() == 0
        pos = batch.positions()
        want, e = R.rope(xv, pos, f, interleaved)
        _within(_np(turned), want, R.rounded(want, e, dtype), "queries")
        vc, vs = R.append(before[2], before[3], np.asarray(vv, np.float64), batch)
        assert np.array_equal(_u8(cache.v), vc) and np.array_equal(cache.v_scale.cpu().numpy(), vs)
        kw, ke = R.rope(kv, pos, f, interleaved)
        kc, ks = R.append(before[0], before[1], kw, batch)
        assert np.array_equal(cache.k_scale.cpu().numpy(), ks) and (_u8(cache.k) != kc).mean() < 1e-3
        # the attention, over the cache and the queries as they are
        held = turned.float().cpu().numpy()
        wy, wl, ye, le = R.attention(held if dtype == "float32" else held.astype(np.float64), _u8(cache.k), ks, vc, vs, batch,
                                     1 / math.sqrt(D))
        _within(_np(y), wy, R.rounded(wy, ye, dtype), "y")
        _within(_np(lse), wl, le, "lse")


def _problem(q, rng, new, lengths, dtype="bfloat16", page=32, H=2, G=4, D=64):
    batch = R.Batch(rng, new, lengths, page)
    cache, codes, scales = _cache(q, rng, batch, H, D)
    x, xv = _as(rng.standard_normal((batch.T, H * G, D)), dtype)
    return batch, cache, codes, scales, x, xv


@pytest.mark.parametrize("dtype,rows", [("bfloat16", 1), ("float32", 1), ("bfloat16", 60), ("float16", 60), ("float32", 60)])
def test_captured_and_replayed_with_other_lengths(cuda_lib, dtype, rows):
    """A decode step (and a chunk) in a graph: lengths, table, offsets and rows change between replays."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(21)
    H, G, D, page, B = 2, 4, 64, 32, 3
    cache = q.KvCache.empty(80, H, page=page, dim=D)
    other = q.KvCache.empty(80, H, page=page, dim=D)
    rope = q.qmm_rope_table(D)
    T = B * rows
    x, k, v = (torch.zeros(T, n, D, device="cuda", dtype=getattr(torch, dtype)) for n in (H * G, H, H))
    table, lengths, offsets = torch.zeros(B, 20, dtype=torch.int32, device="cuda"), _i32([1] * B), _i32(np.arange(B + 1) * rows)
    off = None if rows == 1 else offsets

    def step(c):
        t = q.qmm_kv_append(c, k, v, table, lengths, offsets=off, rope=rope, q=x)
        return q.qmm_kv_attention(c, t, table, lengths, offsets=off, lse=True)
    table.copy_(_i32(rng.permutation(60).reshape(B, 20)))
    lengths.fill_(rows)
    for c in (cache, other):
        step(c), step(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, lse = step(cache)
    for have in ([rows] * B, [rows + 5, rows + 300, rows], [rows + 77, rows + 500, rows + 31]):
        if rows > 1:
            cuts = sorted(rng.integers(0, T + 1, B - 1).tolist())
            offsets.copy_(_i32([0] + cuts + [T - 3]) if cuts[-1] <= T - 3 else _i32([0, 5, 9, T]))
            have = [max(n, int(m)) for n, m in zip(have, (offsets[1:] - offsets[:-1]).tolist())]
        table.copy_(_i32(rng.permutation(80)[:60].reshape(B, 20)))
        lengths.copy_(_i32(have))
        for t, n in ((x, H * G), (k, H), (v, H)):
            t.copy_(_as(rng.standard_normal((T, n, D)), dtype)[0])
        used = T if off is None else int(offsets[-1])
        y.fill_(7), lse.fill_(7)
        graph.replay()
        wy, wl = step(other)
        torch.cuda.synchronize()
        assert q.qmm_device_status() == 0
        assert torch.equal(y[:used], wy[:used]) and torch.equal(lse[:used], wl[:used])
        assert bool((y[used:] == 7).all()) and bool((lse[used:] == 7).all())     # rows behind the last sequence
        assert np.array_equal(_u8(cache.k), _u8(other.k)) and torch.equal(cache.v_scale, other.v_scale)


@pytest.mark.parametrize("new,lengths", [([1, 1], [5000, 3000]), ([200, 150], [900, 2000]), ([4, 4], [30000, 29000])])
def test_two_graphs_of_one_stream_at_once(cuda_lib, new, lengths):
    """Graphs captured on one stream and replayed on two at the same time: each has its partial results to itself."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(22)
    jobs = []
    for _ in range(2):
        batch, cache, _, _, x, _ = _problem(q, rng, new, lengths, page=64, H=4, D=128)
        args = (x, _t(batch.table), _i32(lengths))
        off = None if new == [1, 1] else _t(batch.offsets)
        jobs.append(lambda c=cache, a=args, o=off: q.qmm_kv_attention(c, a[0], a[1], a[2], offsets=o))
    want = [j() for j in jobs]
    graphs, got = [], []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(j())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert q.qmm_device_status() == 0


def test_streams_and_threads(cuda_lib):
    """Calls of several threads, half of them on a stream of their own, the others on one that they share: every result
    that of the call alone, bit for bit."""
    import torch
    q = cuda_lib
    shared = torch.cuda.Stream()
    torch.cuda.synchronize()

    def job(seed):
        rng = np.random.default_rng(seed)
        ps = [_problem(q, rng, [1] * 4, [700, 30, 2000, 1], "bfloat16", D=128), _problem(q, rng, [3, 1], [900, 64], "float32"),
              _problem(q, rng, [150, 80], [800, 80], "float16")]
        rope = q.qmm_rope_table(64)
        pos = _i32(rng.integers(0, 1000, ps[1][4].shape[0]))

        def run():
            out = [q.qmm_rope(ps[1][4], rope, pos)]
            for batch, cache, _, _, x, _ in ps:
                out += q.qmm_kv_attention(cache, x, _t(batch.table), _i32(batch.lengths), offsets=_t(batch.offsets), lse=True)
            return out
        return run
    jobs = [job(30 + i) for i in range(4)]
    want = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st = shared if i % 2 else torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(10):
                got = jobs[i]()
                st.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(want[i], got)):
                    wrong.append(i)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not wrong and q.qmm_device_status() == 0


def test_results_on_another_stream(cuda_lib):
    """stream=: behind work that is still queued on the current one nothing is overwritten or read too early."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(23)
    batch, cache, _, _, x, _ = _problem(q, rng, [1, 1, 1], [300, 40, 1000])
    table, lengths = _t(batch.table), _i32(batch.lengths)
    want = q.qmm_kv_attention(cache, x, table, lengths)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sums = []
    for _ in range(5):
        y = q.qmm_kv_attention(cache, x, table, lengths, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(2_000_000)
        sums.append(y.clone())
        del y
    torch.cuda.synchronize()
    assert all(torch.equal(want, s) for s in sums)


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 2, 40]])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_parts_of_larger_tensors(cuda_lib, new, dtype):
    """Queries and results as parts of larger tensors, heads before rows, odd starts, a table wider than needed with
    rows further apart; nothing beside the results is written."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(24)
    lengths = [300, 45, 700]
    batch, cache, _, _, x, _ = _problem(q, rng, new, lengths, dtype=dtype)
    T, Hq, D = x.shape
    off = None if T == 3 else _t(batch.offsets)
    wide = torch.full((3, batch.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + batch.table.shape[1]] = _t(batch.table)
    table = wide[:, 2:2 + batch.table.shape[1]]
    want = q.qmm_kv_attention(cache, x, _t(batch.table), _i32(lengths), offsets=off)
    for shape, view in (((T, Hq + 3, D + 16), lambda b: b[:, 1:1 + Hq, :D]), ((Hq, T + 2, D), lambda b: b[:, 1:1 + T].transpose(0, 1)),
                        ((T * Hq * D + 1,), lambda b: b[1:].view(T, Hq, D)), ((T, Hq * D + 1), lambda b: b[:, 1:].unflatten(1, (Hq, D)))):
        a, b = (torch.full(shape, 3.0, dtype=x.dtype, device="cuda") for _ in range(2))
        view(a).copy_(x)
        y = q.qmm_kv_attention(cache, view(a), table, _i32(lengths), offsets=off, y=view(b))
        assert torch.equal(y, want)
        view(b).fill_(3.0)
        assert bool((b == 3).all())
    assert q.qmm_device_status() == 0


@pytest.mark.parametrize("dtype,new", [("bfloat16", 1), ("bfloat16", 100), ("float32", 30)])
def test_refused_on_the_device(cuda_lib, dtype, new):
    """Lengths, offsets and pages out of range: reported, the other sequences' results as they should be (not the same
    bits: a sequence that is left out changes where the work of the others is cut)."""
    q = cuda_lib
    rng = np.random.default_rng(25)
    n, lengths = [new] * 3, [300, 200, 250]
    batch, cache, codes, scales, x, xv = _problem(q, rng, n, lengths, dtype=dtype)
    off = None if new == 1 else _t(batch.offsets)
    want, _, e, _ = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 1 / math.sqrt(64))
    e = R.rounded(want, e, dtype)
    for what in ("page", "negative page", "length", "negative length", "offset"):
        table, lens, o = batch.table.copy(), list(lengths), batch.offsets.copy()
        bad = [1]
        if what == "page":
            table[1, 2] = batch.pages
        elif what == "negative page":
            table[1, 0] = -5
        elif what == "length":
            lens[1] = batch.table.shape[1] * 32 + 1
        elif what == "negative length":
            lens[1] = -1
        elif off is None:
            continue
        else:
            o[3], bad = batch.T + 1, [2]
        y = q.qmm_kv_attention(cache, x, _t(table), _i32(lens), offsets=None if off is None else _t(o))
        assert q.qmm_device_status() == q.QMM_EINDEX and q.qmm_device_status() == 0
        for b in range(3):
            if b not in bad:
                rows = slice(batch.offsets[b], batch.offsets[b + 1])
                _within(_np(y)[rows], want[rows], e[rows], f"{what}: sequence {b}")


def test_many_sequences(cuda_lib):
    """More sequences than lanes, warps or blocks; short and empty ones among them."""
    q = cuda_lib
    rng = np.random.default_rng(26)
    B = 700
    lengths = rng.integers(0, 90, B).tolist()
    for dtype, new in (("bfloat16", [1] * B), ("float32", rng.integers(0, 3, B).tolist()), ("bfloat16", rng.integers(0, 40, B).tolist())):
        lens = [max(a, b) for a, b in zip(lengths, new)]
        batch, cache, codes, scales, x, xv = _problem(q, rng, new, lens, dtype=dtype, page=16, H=1, G=2, D=32)
        off = None if new == [1] * B else _t(batch.offsets)
        y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _i32(lens), offsets=off, lse=True)
        assert q.qmm_device_status() == 0
        wy, wl, ye, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 1 / math.sqrt(32))
        _within(_np(y), wy, R.rounded(wy, ye, dtype), "y")
        _within(_np(lse), wl, le, "lse")
        k, kv = _as(rng.standard_normal((batch.T, 1, 32)), dtype)
        q.qmm_kv_append(cache, k, k, _t(batch.table), _i32(lens), offsets=off)
        want, ws = R.append(codes[0], scales[0], np.asarray(kv, np.float64), batch)
        assert np.array_equal(_u8(cache.k), want) and np.array_equal(cache.k_scale.cpu().numpy(), ws)
    assert q.qmm_device_status() == 0


@pytest.mark.parametrize("dtype,new,length", [("bfloat16", 1, 60000), ("bfloat16", 10, 60000), ("float32", 20, 9000), ("float32", 3, 60000), ("bfloat16", 300, 60000), ("float16", 300, 60000)])
def test_expired_wait_is_reported_and_the_next_call_is_right(cuda_lib, dtype, new, length):
    """The copies of the first block stop after one tile: the waits for the next one run out, the kernel says so, frees
    what it holds and returns; the next call finds everything in order."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(27)
    batch, cache, _, _, x, _ = _problem(q, rng, [new], [length], dtype=dtype, page=128, H=8, G=2, D=64)
    args = (x, _t(batch.table), _i32([length]))
    off = None if new == 1 else _t(batch.offsets)
    want = q.qmm_kv_attention(cache, *args, offsets=off)
    assert q.qmm_device_status() == 0
    assert q.inject_stall(1) == 0
    q.qmm_kv_attention(cache, *args, offsets=off)
    assert q.qmm_device_status() == q.QMM_ETIMEOUT and q.qmm_device_status() == 0
    for _ in range(2):
        assert torch.equal(q.qmm_kv_attention(cache, *args, offsets=off), want)
    assert q.qmm_device_status() == 0 and q.inject_stall(0) == 0


def test_repeated_calls_agree_bit_for_bit(cuda_lib):
    import torch
    q = cuda_lib
    rng = np.random.default_rng(28)
    for dtype, new, lengths in (("bfloat16", [1, 1], [20000, 7]), ("bfloat16", [300, 100], [3000, 100]), ("float32", [9], [5000]),
                                ("bfloat16", [5], [90000]), ("float16", [3, 4], [50000, 40000]), ("float32", [99], [3000])):
        batch, cache, _, _, x, _ = _problem(q, rng, new, lengths, dtype=dtype, page=64, H=2, G=4, D=128)
        args = (x, _t(batch.table), _i32(lengths))
        off = None if new == [1, 1] else _t(batch.offsets)
        first = q.qmm_kv_attention(cache, *args, offsets=off, lse=True)
        for _ in range(20):
            again = q.qmm_kv_attention(cache, *args, offsets=off, lse=True)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_past_32_bits(cuda_lib):
    """A cache whose codes and rows lie more than 2^32 bytes from its beginning."""
    import torch
    q = cuda_lib
    H, D, page = 16, 256, 128
    pages = (1 << 32) // (H * D * page) + 40                     # 8 KB a token
    cache = q.KvCache.empty(pages, H, page=page, dim=D)
    rng = np.random.default_rng(29)
    lengths = [300]
    batch = R.Batch(rng, [300], lengths, page)
    batch.table = np.array([[pages - 1, pages - 7, pages - 3]], np.int32)
    small = R.Batch(rng, [300], lengths, page)
    small.table = np.array([[2, 1, 0]], np.int32)
    twin = q.KvCache.empty(3, H, page=page, dim=D)
    x, k, v = (_as(rng.standard_normal((300, n, D)), "bfloat16")[0] for n in (H, H, H))
    for c, b in ((cache, batch), (twin, small)):
        q.qmm_kv_append(c, k, v, _t(b.table), _i32(lengths), offsets=_t(b.offsets))
    big = torch.empty(300, H, (1 << 32) // (2 * 300 * H) // 8 * 8 + 4096, device="cuda", dtype=torch.bfloat16)[:, :, -D:]
    big.copy_(x)
    for rows in (300, 1):
        got, want = (q.qmm_kv_attention(c, a[-rows:], _t(b.table), _i32(lengths), offsets=None if rows == 1 else _t(b.offsets))
                     for c, b, a in ((cache, batch, big), (twin, small, x)))
        assert torch.equal(got, want)
    assert q.qmm_device_status() == 0

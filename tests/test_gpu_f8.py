"""The block-scaled 8-bit-float operators on the GPU against the 64-bit reference (f8_reference.py): sizes from one
token up, odd and ragged ones, every value type, row pitches, empty groups, values that are not finite, refusals."""
import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _as(a, dtype):
    """float32 numpy values -> (device tensor of dtype, the float32 values it holds)."""
    import torch
    t = _t(np.asarray(a, np.float32)).to(getattr(torch, dtype))
    return t, t.float().cpu().numpy()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _x(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    return x * np.where(rng.random((M, K)) < 0.01, 20, 1).astype(np.float32)


def _close(got, want, e, dtype, what=""):
    b = R.out_bound(want, e, dtype)
    bad = ~(np.abs(got - want) <= b)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst {np.nanmax(np.abs(got - want) / b):.3g} bounds"


def _padded(t, pad, skip=0):
    """The same values in rows `pad` further apart, starting `skip` elements into the buffer."""
    import torch
    M, K = t.shape
    buf = torch.full((M * (K + pad) + skip + pad,), 7.0, dtype=t.dtype, device=t.device)
    v = buf.as_strided((M, K), (K + pad, 1), skip)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,pad,skip", [(1, 1, 0, 0), (3, 127, 0, 0), (5, 128, 3, 1), (2, 129, 0, 0), (7, 640, 8, 0),
                                          (4, 1000, 0, 0), (33, 516, 4, 4), (1000, 272, 0, 0), (2, 65536 + 4, 1, 3)])
def test_quantize_bitwise(cuda_lib, dtype, M, K, pad, skip):
    x, xv = _as(_x(np.random.default_rng(M + K), M, K), dtype)
    c, s = cuda_lib.qmm_f8_quantize(_padded(x, pad, skip))
    codes, scales = R.quantize(xv)
    import torch
    assert np.array_equal(c.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))


def test_quantize_extremes(cuda_lib):
    """Zero blocks, subnormals, the largest floats; a block with a NaN or an infinity keeps neither finite codes where x
    is not finite nor a finite scale."""
    x = np.zeros((7, 256), np.float32)
    x[1] = 1e-41
    x[2] = np.linspace(-3e38, 3e38, 256)
    x[3] = np.linspace(-1e-38, 1e-38, 256)
    x[4, 5] = np.nan
    x[5, 200] = np.inf
    x[6] = -0.0
    import torch
    c, s = cuda_lib.qmm_f8_quantize(_t(x))
    codes, scales = R.quantize(x)
    c, s = c.view(torch.uint8).cpu().numpy(), s.cpu().numpy()
    fine = np.isfinite(scales)
    assert np.array_equal(s[fine], scales[fine]) and np.isnan(s[4, 0]) and np.isinf(s[5, 1])
    same = np.repeat(fine, 128, 1)
    assert np.array_equal(c[same], codes[same])
    assert c[4, 5] & 0x7f == 0x7f and c[5, 200] & 0x7f == 0x7f


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 300, 2048), (2, 64, 112), (3, 129, 144), (8, 1000, 1152), (16, 256, 384),
          (17, 100, 1040), (31, 2050, 256), (33, 300, 512), (64, 127, 5120), (65, 128, 2064), (129, 257, 272),
          (255, 130, 128), (257, 1, 640), (300, 640, 1152), (513, 1000, 400), (1030, 5000, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_shapes(cuda_lib, M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    W, S = R.weights(rng, N, K)
    for i, dtype in enumerate(TYPES):
        if M * N * K > 1 << 28 and dtype == "float16":
            continue
        x, xv = _as(_x(rng, M, K), dtype)
        before = cuda_lib.qmm_launch_count()
        y = cuda_lib.qmm_f8(_t(W), _t(S), x)
        assert cuda_lib.qmm_launch_count() - before == (1 if M <= 16 else 2)
        assert cuda_lib.qmm_device_status() == 0
        assert str(y.dtype) == "torch." + dtype and tuple(y.shape) == (M, N)
        want, A = R.product(W, S, xv)
        _close(_np(y), want, R.bound(K, A), dtype, f"{M}x{N}x{K} {dtype}")


@pytest.mark.parametrize("M,N,K,launches", [(1, 14336, 4096, 2), (6, 1024, 5120, 1), (13, 5120, 5120, 2),
                                            (1, 25600, 4096, 2), (16, 5120, 17408, 2), (5, 17408, 17408, 2),
                                            (100, 14336, 4096, 2), (64, 5120, 5120, 2), (300, 14336, 1024, 2)])
def test_product_full_size_matrices(cuda_lib, M, N, K, launches):
    """Matrices of the size a model has, on sampled columns: few rows with x quantised inside the product and, above
    the size it can do that for, in front of it."""
    import torch
    rng = np.random.default_rng(N + K + M)
    g = torch.Generator(device="cuda").manual_seed(M)
    W = torch.randint(0, 0x70, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    W |= torch.randint(0, 2, (N, K), generator=g, device="cuda", dtype=torch.uint8) << 7
    S = torch.rand(-(-N // 128), -(-K // 128), generator=g, device="cuda") * 1e-3
    x, xv = _as(_x(rng, M, K), "bfloat16")
    before = cuda_lib.qmm_launch_count()
    y = cuda_lib.qmm_f8(W, S, x, dtype=torch.float32)
    assert cuda_lib.qmm_launch_count() - before == launches
    assert cuda_lib.qmm_device_status() == 0
    blocks = np.unique(np.concatenate([[0, -(-N // 128) - 1], rng.integers(0, -(-N // 128), 6)]))
    for b in blocks:
        n = slice(128 * b, min(128 * b + 128, N))
        want, A = R.product(W[n].cpu().numpy(), S[b:b + 1].cpu().numpy(), xv)
        _close(_np(y[:, n]), want, R.bound(K, A), "float32", f"block {b}")


@pytest.mark.parametrize("xt,yt", [(a, b) for a in TYPES for b in TYPES if a != b])
def test_product_types_and_pitches(cuda_lib, xt, yt):
    import torch
    rng = np.random.default_rng(5)
    for M, N, K, px, py, skip in ((5, 200, 272, 3, 5, 1), (40, 131, 128, 8, 0, 0), (300, 257, 144, 0, 7, 3)):
        W, S = R.weights(rng, N, K)
        x, xv = _as(_x(rng, M, K), xt)
        y = _padded(torch.zeros((M, N), dtype=getattr(torch, yt), device="cuda"), py, skip)
        base = y._base if y._base is not None else y
        out = cuda_lib.qmm_f8(_t(W), _t(S), _padded(x, px, skip), y=y)
        assert out is y
        want, A = R.product(W, S, xv)
        _close(_np(y), want, R.bound(K, A), yt, f"{xt} {yt}")
        # nothing between the rows is written
        keep = torch.ones(base.numel(), dtype=torch.bool, device="cuda")
        keep.as_strided((M, N), (N + py, 1), skip)[:] = False
        assert torch.all(base.reshape(-1)[keep] == 7.0)


def test_product_of_a_vector_and_empty(cuda_lib):
    import torch
    rng = np.random.default_rng(1)
    W, S = R.weights(rng, 70, 160)
    x = _t(_x(rng, 1, 160))
    assert torch.equal(cuda_lib.qmm_f8(_t(W), _t(S), x[0]), cuda_lib.qmm_f8(_t(W), _t(S), x))
    assert tuple(cuda_lib.qmm_f8(_t(W), _t(S), x[:0]).shape) == (0, 70)
    y = cuda_lib.qmm_f8(torch.zeros((9, 0), dtype=torch.uint8, device="cuda"), torch.zeros((1, 0), device="cuda"),
                        torch.zeros((4, 0), device="cuda"))
    assert tuple(y.shape) == (4, 9) and not y.any()


def test_product_large_magnitudes_and_zeros(cuda_lib):
    rng = np.random.default_rng(2)
    M, N, K = 20, 140, 400
    W, S = R.weights(rng, N, K)
    x = _x(rng, M, K) * (10.0 ** rng.integers(-30, 30, (M, 1))).astype(np.float32)
    x[3] = 0
    y = cuda_lib.qmm_f8(_t(W), _t(S), _t(x))
    want, A = R.product(W, S, x)
    _close(_np(y), want, R.bound(K, A), "float32")
    assert not y[3].any()


def test_product_not_finite(cuda_lib):
    """A NaN or infinity of x makes its own row NaN, a NaN code of W its own column; nothing else changes."""
    rng = np.random.default_rng(3)
    M, N, K = 40, 200, 384
    W, S = R.weights(rng, N, K)
    x = _x(rng, M, K)
    want, A = R.product(W, S, x)
    x[7, 300] = np.nan
    x[11, 0] = np.inf
    W2 = W.copy()
    W2[150, 5] = 0x7f
    y = _np(cuda_lib.qmm_f8(_t(W2), _t(S), _t(x)))
    assert np.isnan(y[[7, 11]]).all() and np.isnan(y[:, 150]).all()
    rows, cols = [i for i in range(M) if i not in (7, 11)], [i for i in range(N) if i != 150]
    _close(y[np.ix_(rows, cols)], want[np.ix_(rows, cols)], R.bound(K, A)[np.ix_(rows, cols)], "float32")


@pytest.mark.parametrize("M,N,K", [(3, 1000, 4096), (200, 2600, 1040), (700, 1500, 2048)])
def test_product_repeats_bit_for_bit(cuda_lib, M, N, K):
    """Also on another stream and out of a replayed graph."""
    import torch
    rng = np.random.default_rng(M)
    W, S = (_t(a) for a in R.weights(rng, N, K))
    x = _t(_x(rng, M, K)).bfloat16()
    y = cuda_lib.qmm_f8(W, S, x, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(y, cuda_lib.qmm_f8(W, S, x, dtype=torch.float32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = torch.empty_like(y)
    cuda_lib.qmm_f8(W, S, x, y=z, stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    z.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cuda_lib.qmm_f8(W, S, x, y=z, stream=side)
    for _ in range(3):
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_product_two_streams_at_once(cuda_lib):
    import torch
    rng = np.random.default_rng(9)
    W, S = (_t(a) for a in R.weights(rng, 900, 1024))
    xs = [_t(_x(rng, m, 1024)) for m in (5, 260)]
    want = [cuda_lib.qmm_f8(W, S, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(cuda_lib.qmm_f8(W, S, xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])


# ---------------------------------------------------------------------------
# Grouped by expert
# ---------------------------------------------------------------------------
def _experts(rng, E, N, K):
    parts = [R.weights(rng, N, K) for _ in range(E)]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


GROUPS = [([1], 128, 128), ([0, 5, 0], 100, 272), ([17, 0, 1, 40], 257, 400), ([0, 0, 3], 64, 1024),
          ([300, 2, 0, 129, 16], 130, 144), ([1] * 64, 200, 256), ([5, 0, 9] * 20, 129, 128), ([700, 0, 33], 384, 640),
          ([0] * 299 + [4], 32, 16), ([2, 0, 0, 1] * 256, 16, 32)]


@pytest.mark.parametrize("sizes,N,K", GROUPS)
@pytest.mark.parametrize("gather", [False, True])
def test_experts(cuda_lib, sizes, N, K, gather):
    rng = np.random.default_rng(len(sizes) * 31 + N + K)
    E, total = len(sizes), sum(sizes)
    W, S = _experts(rng, E, N, K)
    dtype = TYPES[(N + K) % 3]
    M = max(1, total // 2) if gather else total
    x, xv = _as(_x(rng, M, K), dtype)
    rows = rng.integers(0, M, total).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = cuda_lib.qmm_f8_experts(_t(W), _t(S), x, _t(offsets), rows=_t(rows) if gather else None)
    assert cuda_lib.qmm_device_status() == 0
    src = xv[rows] if gather else xv
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        if sizes[e]:
            want, A = R.product(W[e], S[e], src[r])
            _close(_np(y[r]), want, R.bound(K, A), dtype, f"expert {e}")


def test_experts_no_rows_and_spare_rows(cuda_lib):
    """Rows of y past the last group keep what they held, also when every group is empty."""
    import torch
    rng = np.random.default_rng(4)
    W, S = (_t(a) for a in _experts(rng, 3, 140, 256))
    x = _t(_x(rng, 50, 256))
    y = torch.full((50, 140), 7.0, device="cuda")
    cuda_lib.qmm_f8_experts(W, S, x, torch.zeros(4, dtype=torch.int32, device="cuda"), y=y)
    assert torch.all(y == 7)
    rows = torch.full((50,), 1 << 30, dtype=torch.int32, device="cuda")   # only the first 20 are looked at
    rows[:20] = torch.arange(20, device="cuda")
    cuda_lib.qmm_f8_experts(W, S, x, _t(np.array([0, 0, 13, 20], np.int32)), rows=rows, y=y)
    assert cuda_lib.qmm_device_status() == 0
    assert torch.all(y[20:] == 7)
    assert torch.equal(y[:13], cuda_lib.qmm_f8(W[1], S[1], x[:13]))


def test_experts_bad_indices_are_reported(cuda_lib):
    """Row indices and offsets out of range: skipped by the kernels' own checks, reported, and the next call is whole."""
    import torch
    rng = np.random.default_rng(6)
    W, S = (_t(a) for a in _experts(rng, 2, 140, 256))
    x = _t(_x(rng, 30, 256))
    offsets = _t(np.array([0, 10, 30], np.int32))
    good = cuda_lib.qmm_f8_experts(W, S, x, offsets)
    rows = torch.arange(30, dtype=torch.int32, device="cuda")
    rows[3], rows[25] = -1, 30
    y = cuda_lib.qmm_f8_experts(W, S, x, offsets, rows=rows)
    assert cuda_lib.qmm_device_status() == cuda_lib.QMM_EINDEX
    keep = [i for i in range(30) if i not in (3, 25)]
    assert torch.equal(y[keep], good[keep])
    for bad in ([0, 31, 31], [-1, 10, 30], [0, 20, 10], [0, 1 << 30, 30]):
        cuda_lib.qmm_f8_experts(W, S, x, _t(np.array(bad, np.int32)))
        assert cuda_lib.qmm_device_status() == cuda_lib.QMM_EINDEX, bad
    assert cuda_lib.qmm_device_status() == 0
    assert torch.equal(good, cuda_lib.qmm_f8_experts(W, S, x, offsets))


def test_experts_graph_replays_with_other_groups(cuda_lib):
    import torch
    rng = np.random.default_rng(8)
    W, S = (_t(a) for a in _experts(rng, 4, 150, 384))
    x = _t(_x(rng, 90, 384)).half()
    offsets = torch.zeros(5, dtype=torch.int32, device="cuda")
    y = torch.empty((90, 150), dtype=torch.float16, device="cuda")
    st = torch.cuda.Stream()
    cuda_lib.qmm_f8_experts(W, S, x, offsets, y=y, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        cuda_lib.qmm_f8_experts(W, S, x, offsets, y=y, stream=st)
    for groups in ([0, 90, 90, 90, 90], [0, 1, 2, 45, 90], [0, 0, 0, 0, 90]):
        offsets.copy_(_t(np.array(groups, np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        for e in range(4):
            a, b = groups[e], groups[e + 1]
            if b > a:
                want, A = R.product(W[e].cpu().numpy(), S[e].cpu().numpy(), x[a:b].float().cpu().numpy())
                _close(_np(y[a:b]), want, R.bound(384, A), "float16")


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------
def _check_route(r, x, k, score, normalize, factor=1.0):
    w, e, off, rows, slots = R.route(x, k, score, normalize, factor)
    assert np.array_equal(r.experts.cpu().numpy(), e)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    # exp to two ulp at most on an argument rounded once (|argument| <= 104 where exp is not 0), E terms summed in
    # fp32 (at most 37 roundings on a path), a division and two products
    got, n = r.weights.cpu().numpy(), 37 + 2 + 104 + 3
    assert np.all(np.abs(got - w) <= n * 2.0 ** -24 * np.abs(w) * 2 + 1e-37), np.abs(got - w).max()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (8, 128, 8), (17, 33, 32), (127, 64, 6), (128, 200, 4),
                                   (129, 7, 2), (300, 1024, 32), (1000, 512, 10), (2050, 60, 6), (5000, 4, 1)])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route(cuda_lib, T, E, k, score, normalize):
    rng = np.random.default_rng(T + E + k)
    dtype = TYPES[(T + E) % 3]
    x, xv = _as(rng.standard_normal((T, E)) * 3, dtype)
    before = cuda_lib.qmm_launch_count()
    r = cuda_lib.qmm_route(_padded(x, T % 4, T % 2), k, score=score, normalize=normalize, factor=2.5)
    assert cuda_lib.qmm_launch_count() - before == (1 if T <= 128 else 2)
    _check_route(r, xv, k, score, normalize, 2.5)


@pytest.mark.parametrize("T,E,k,launches", [(10241, 33, 3, 2), (30001, 64, 6, 3), (70000, 100, 2, 3), (12000, 1024, 4, 3)])
def test_route_many_tokens(cuda_lib, T, E, k, launches):
    rng = np.random.default_rng(T)
    x, xv = _as(rng.standard_normal((T, E)) * 2 + rng.standard_normal(E), "bfloat16")
    before = cuda_lib.qmm_launch_count()
    r = cuda_lib.qmm_route(x, k)
    assert cuda_lib.qmm_launch_count() - before == launches
    _check_route(r, xv, k, "softmax", True)


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_masks_and_nan(cuda_lib, T, score):
    """Equal logits, +0 and -0, masked experts (-inf and the lowest float), NaN, a row with nothing left."""
    rng = np.random.default_rng(T)
    E, k = 40, 6
    x = rng.integers(-2, 3, (T, E)).astype(np.float32)
    x[x == 0] *= rng.choice([-1, 1], (x == 0).sum())
    x[:, 3] = -np.inf
    x[:, 9] = np.finfo(np.float32).min
    x[::3, 11] = np.nan
    x[0] = -np.inf
    x[-1, 4:] = -np.inf
    r = cuda_lib.qmm_route(_t(x), k, score=score)
    _check_route(r, x, k, score, True)
    assert not r.weights[0].any()


def test_route_of_no_tokens(cuda_lib):
    import torch
    r = cuda_lib.qmm_route(torch.zeros((0, 6), device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 7 and r.weights.shape == (0, 2)


# ---------------------------------------------------------------------------
# The expert layer
# ---------------------------------------------------------------------------
def _moe_reference(x, w, e, offsets, slots, Wg, Sg, Wu, Su, Wd, Sd):
    T, k = e.shape
    y, b = np.zeros((T, Wd.shape[1])), np.zeros((T, Wd.shape[1]))
    for j in range(k):
        for ex in np.unique(e[:, j]):
            t = np.nonzero(e[:, j] == ex)[0]
            h, eh = R.gated(Wg[ex], Sg[ex], Wu[ex], Su[ex], x[t])
            d, bd = R.down_product(Wd[ex], Sd[ex], h, eh)
            y[t] += w[t, j:j + 1] * d
            b[t] += w[t, j:j + 1] * (bd + (k + 1) * 2.0 ** -24 * (np.abs(d) + bd))
    return y, b


@pytest.mark.parametrize("T,k,E,H,I,dtype", [(1, 1, 1, 16, 16, "float32"), (1, 2, 8, 256, 128, "bfloat16"),
                                             (4, 6, 16, 272, 144, "float16"), (33, 2, 3, 144, 272, "bfloat16"),
                                             (60, 4, 40, 128, 80, "float32"), (200, 3, 6, 400, 384, "float16"),
                                             (520, 2, 4, 128, 256, "bfloat16"), (129, 8, 128, 64, 48, "float16")])
def test_moe(cuda_lib, T, k, E, H, I, dtype):
    rng = np.random.default_rng(T + k + E + H + I)
    Wg, Sg = _experts(rng, E, I, H)
    Wu, Su = _experts(rng, E, I, H)
    Wd, Sd = _experts(rng, E, H, I)
    x, xv = _as(_x(rng, T, H), dtype)
    logits = rng.standard_normal((T, E)).astype(np.float32) + rng.standard_normal(E).astype(np.float32)
    r = cuda_lib.qmm_route(_t(logits), k)
    before = cuda_lib.qmm_launch_count()
    y = cuda_lib.qmm_f8_moe(x, r, *(_t(a) for a in (Wg, Sg, Wu, Su, Wd, Sd)))
    assert cuda_lib.qmm_launch_count() - before == 4
    assert cuda_lib.qmm_device_status() == 0
    want, b = _moe_reference(xv, r.weights.cpu().numpy().astype(np.float64), r.experts.cpu().numpy(), None, None,
                             Wg, Sg, Wu, Su, Wd, Sd)
    _close(_np(y), want, b, dtype)
    import torch
    again = cuda_lib.qmm_f8_moe(x, r, *(_t(a) for a in (Wg, Sg, Wu, Su, Wd, Sd)))
    assert torch.equal(y, again)


def test_moe_empty(cuda_lib):
    import torch
    rng = np.random.default_rng(0)
    W = [_t(a) for a in (*_experts(rng, 2, 32, 64), *_experts(rng, 2, 32, 64), *_experts(rng, 2, 64, 32))]
    r = cuda_lib.qmm_route(torch.zeros((0, 2), device="cuda"), 1)
    assert tuple(cuda_lib.qmm_f8_moe(torch.zeros((0, 64), device="cuda"), r, *W).shape) == (0, 64)


def test_moe_bad_slots_are_reported(cuda_lib):
    import torch
    rng = np.random.default_rng(0)
    W = [_t(a) for a in (*_experts(rng, 2, 32, 64), *_experts(rng, 2, 32, 64), *_experts(rng, 2, 64, 32))]
    x = _t(_x(rng, 5, 64))
    r = cuda_lib.qmm_route(_t(rng.standard_normal((5, 2)).astype(np.float32)), 1)
    good = cuda_lib.qmm_f8_moe(x, r, *W)
    slots = r.slots.clone()
    slots[2] = 5
    cuda_lib.qmm_f8_moe(x, r._replace(slots=slots), *W)
    assert cuda_lib.qmm_device_status() == cuda_lib.QMM_EINDEX
    assert torch.equal(good, cuda_lib.qmm_f8_moe(x, r, *W))
    assert cuda_lib.qmm_device_status() == 0


def test_example_layer_agrees_with_grouped_products(cuda_lib):
    """The layer against its parts: bf16 rounding of the result (2^-9 of it) and of h, whose codes (2^-4 apart) differ
    where the two SiLUs fall on different sides of a boundary: rarely, so far below 1 % of the norm."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "f8_expert_layer.py")
    spec = importlib.util.spec_from_file_location("f8_expert_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for args in ((1, 8, 2, 256, 128), (64, 32, 4, 512, 272), (700, 5, 2, 384, 256)):
        assert example.main(*args) < 1e-2


# ---------------------------------------------------------------------------
# Failure detection and refusals
# ---------------------------------------------------------------------------
def test_stalled_copies_are_reported(cuda_lib):
    """A copy that never comes: the waits run out, the call is reported, the next one is whole."""
    import torch
    rng = np.random.default_rng(0)
    W, S = (_t(a) for a in R.weights(rng, 600, 2048))
    x = _t(_x(rng, 20, 2048))
    y = cuda_lib.qmm_f8(W, S, x)
    cuda_lib.inject_stall(1)
    cuda_lib.qmm_f8(W, S, x)
    assert cuda_lib.qmm_device_status() == cuda_lib.QMM_ETIMEOUT
    assert cuda_lib.qmm_device_status() == 0
    assert torch.equal(y, cuda_lib.qmm_f8(W, S, x))


def test_binding_refusals(cuda_lib):
    import torch
    q = cuda_lib
    W = torch.zeros((4, 32), dtype=torch.uint8, device="cuda")
    S = torch.ones((1, 1), device="cuda")
    x = torch.zeros((2, 32), device="cuda")
    for bad in (lambda: q.qmm_f8(W.float(), S, x), lambda: q.qmm_f8(W[:, ::2], S, x), lambda: q.qmm_f8(W, S.half(), x),
                lambda: q.qmm_f8(W, S[0], x), lambda: q.qmm_f8(W, S, x[:, :16]), lambda: q.qmm_f8(W, S, x.double()),
                lambda: q.qmm_f8(W, S, x.t()), lambda: q.qmm_f8(W, S, x, y=torch.zeros((2, 5), device="cuda")),
                lambda: q.qmm_f8(W, S, x, dtype=torch.int8), lambda: q.qmm_f8(W.cpu(), S, x),
                lambda: q.qmm_route(x, 2, score="tanh"), lambda: q.qmm_f8_quantize(x.int()),
                lambda: q.qmm_f8_experts(W[None], S[None], x, torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: q.qmm_f8_experts(W[None], S[None], x, torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.QmmError):
        q.qmm_f8(torch.zeros((4, 24), dtype=torch.uint8, device="cuda"), S, x[:, :24])
    with pytest.raises(q.QmmError):
        q.qmm_f8(W, S, x[:1].expand(3, 32))
    with pytest.raises(q.QmmError):
        q.qmm_route(x, 33)

"""The 8-bit-float products on shapes that cut and deal out their tiles in every way (f8_shapes.py), on sampled rows and
columns; values that are not finite, and copies that never come, in every kernel."""
import numpy as np
import pytest

import f8_reference as R
import f8_shapes as shapes

pytestmark = pytest.mark.gpu


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(got, want, e, what=""):
    b = R.out_bound(want, e, "float32")
    bad = ~(np.abs(got - want) <= b)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst {np.nanmax(np.abs(got - want) / b):.3g} bounds"


def _matrices(g, E, N, K, size):
    """Codes of every finite value up to 240 and scales for products of about `size`, made on the GPU."""
    import torch
    W = torch.randint(0, 0x78, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)
    W |= torch.randint(0, 2, (E, N, K), generator=g, device="cuda", dtype=torch.uint8) << 7
    # a code's mean square: codes are spread over fifteen binades, the top ones count
    s = size / (58.0 * K ** 0.5)
    S = torch.rand(E, -(-N // 128), -(-K // 128), generator=g, device="cuda") * s + s / 2
    return W, S


def _x(g, M, K):
    import torch
    x = torch.randn(M, K, generator=g, device="cuda")
    return (x * (1 + 19 * (torch.rand(M, K, generator=g, device="cuda") < 0.01))).bfloat16()


def _some(rng, n, most):
    return np.arange(n) if n <= most else np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, most)]))


def _check_columns(rng, y, W, S, xv, rows, what=""):
    """Sampled column blocks of y[rows] against the 64-bit product; the first and the last among them."""
    N, K = W.shape
    for b in _some(rng, -(-N // 128), 5):
        n = slice(128 * b, min(128 * b + 128, N))
        want, A = R.product(W[n].cpu().numpy(), S[b:b + 1].cpu().numpy(), xv)
        _close(_np(y[rows][:, n]), want, R.bound(K, A), f"{what} block {b}")


@pytest.mark.parametrize("M,N,K,launches,tokens,cols,G,step,rule", shapes.ONE_MATRIX)
def test_one_matrix(cuda_lib, M, N, K, launches, tokens, cols, G, step, rule):
    import torch
    rng = np.random.default_rng(M + N + K)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    W, S = _matrices(g, 1, N, K, 1.0)
    x = _x(g, M, K)
    before = cuda_lib.qmm_launch_count()
    y = cuda_lib.qmm_f8(W[0], S[0], x, dtype=torch.float32)
    assert cuda_lib.qmm_launch_count() - before == launches
    assert cuda_lib.qmm_device_status() == 0
    rows = _t(_some(rng, M, 40))
    _check_columns(rng, y, W[0], S[0], x[rows].float().cpu().numpy(), rows)
    assert not y.isnan().any()
    for _ in range(3):
        assert torch.equal(y, cuda_lib.qmm_f8(W[0], S[0], x, dtype=torch.float32))


@pytest.mark.parametrize("sizes,N,K,tokens,cols,G,step,rule", shapes.EXPERTS)
def test_experts(cuda_lib, sizes, N, K, tokens, cols, G, step, rule):
    import torch
    rng = np.random.default_rng(N + K)
    g = torch.Generator(device="cuda").manual_seed(N)
    E, total = len(sizes), sum(sizes)
    W, S = _matrices(g, E, N, K, 1.0)
    x = _x(g, total // 2 + 1, K)
    rows = torch.randint(0, len(x), (total,), generator=g, device="cuda", dtype=torch.int32)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    y = cuda_lib.qmm_f8_experts(W, S, x, _t(offsets.astype(np.int32)), rows=rows, dtype=torch.float32)
    assert cuda_lib.qmm_device_status() == 0
    used = [e for e in range(E) if sizes[e]]
    for e in [used[i] for i in _some(rng, len(used), 4)]:
        at = _t(offsets[e] + _some(rng, sizes[e], 20))
        _check_columns(rng, y, W[e], S[e], x[rows[at].long()].float().cpu().numpy(), at, f"expert {e}")
    assert not y.isnan().any()
    assert torch.equal(y, cuda_lib.qmm_f8_experts(W, S, x, _t(offsets.astype(np.int32)), rows=rows, dtype=torch.float32))


def _layer(g, T, k, E, H, I):
    """A route whose choices go round the experts, and the weights of a layer."""
    import torch
    pairs = torch.arange(T * k, device="cuda").view(T, k) % E
    flat = pairs.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    return w, pairs, offsets, order // k, slots.view(T, k), [*_matrices(g, E, I, H, 1.0), *_matrices(g, E, I, H, 1.0),
                                                             *_matrices(g, E, H, I, 1.0)]


def _route(q, w, pairs, offsets, rows, slots):
    import torch
    i32 = torch.int32
    return q.Route(w, pairs.to(i32), offsets, rows.to(i32), slots.to(i32))


@pytest.mark.parametrize("T,k,E,H,I,gate_up,down", shapes.EXPERT_LAYERS)
def test_expert_layers(cuda_lib, T, k, E, H, I, gate_up, down):
    import torch
    rng = np.random.default_rng(T + H)
    g = torch.Generator(device="cuda").manual_seed(T)
    *r, mlp = _layer(g, T, k, E, H, I)
    x = _x(g, T, H)
    y = cuda_lib.qmm_f8_moe(x, _route(cuda_lib, *r), *mlp, dtype=torch.float32)
    assert cuda_lib.qmm_device_status() == 0
    w, pairs = r[0].cpu().numpy().astype(np.float64), r[1].cpu().numpy()
    tokens = _some(rng, T, 6)
    xv = x[_t(tokens)].float().cpu().numpy()
    want, bound = np.zeros((len(tokens), H)), np.zeros((len(tokens), H))
    for e in np.unique(pairs[tokens]):
        Wg, Sg, Wu, Su, Wd, Sd = (t[e].cpu().numpy() for t in mlp)
        for j in range(k):
            i = np.nonzero(pairs[tokens, j] == e)[0]
            if len(i):
                h, eh = R.gated(Wg, Sg, Wu, Su, xv[i])
                d, bd = R.down_product(Wd, Sd, h, eh)
                c = w[tokens[i], j:j + 1]
                want[i] += c * d
                bound[i] += c * (bd + (k + 1) * 2.0 ** -24 * (np.abs(d) + bd))
    _close(_np(y)[tokens], want, bound)
    # the bound allows for codes on a boundary; as a whole the result is much closer
    assert np.linalg.norm(_np(y)[tokens] - want) < 1e-2 * np.linalg.norm(want)
    assert torch.equal(y, cuda_lib.qmm_f8_moe(x, _route(cuda_lib, *r), *mlp, dtype=torch.float32))


# ---------------------------------------------------------------------------
# Values that are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", [(5, 200, 384), (300, 700, 384), (300, 700, 4096)])
def test_not_finite_in_one_matrix(cuda_lib, M, N, K):
    """A NaN or infinity of x makes its own row NaN, a NaN code of W its own column; nothing else changes."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    W, S = (t[0] for t in _matrices(g, 1, N, K, 1.0))
    x = _x(g, M, K).float()
    want = cuda_lib.qmm_f8(W, S, x)
    x[1, 300], x[M - 1, 0] = torch.nan, torch.inf
    W[150, 5], W[N - 1, K - 1] = 0x7f, 0xff
    y = cuda_lib.qmm_f8(W, S, x)
    nan = torch.zeros_like(y, dtype=torch.bool)
    nan[[1, M - 1]], nan[:, [150, N - 1]] = True, True
    assert torch.equal(y.isnan(), nan) and torch.equal(y[~nan], want[~nan])


@pytest.mark.parametrize("T,E", [(6, 4), (300, 4)])          # the kernel for few rows of an expert, for many
def test_not_finite_in_an_expert_layer(cuda_lib, T, E):
    """x: its token; W_gate or W_up: the tokens of the expert (one scale block of h); W_down: a column of those; a row of
    the grouped product: itself."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    H, I, k = 272, 144, 2
    *r, mlp = _layer(g, T, k, E, H, I)
    route, x = _route(cuda_lib, *r), _x(g, T, H).float()
    want = cuda_lib.qmm_f8_moe(x, route, *mlp)
    rows = cuda_lib.qmm_f8_experts(mlp[0], mlp[1], x, route.offsets, rows=route.rows)
    bad = x.clone()
    bad[1, 7], bad[T - 1, H - 1] = torch.inf, torch.nan
    hit = torch.zeros(T, dtype=torch.bool, device="cuda")
    hit[[1, T - 1]] = True
    y = cuda_lib.qmm_f8_moe(bad, route, *mlp)
    assert torch.equal(y.isnan(), hit[:, None].expand_as(y)) and torch.equal(y[~hit], want[~hit])
    y = cuda_lib.qmm_f8_experts(mlp[0], mlp[1], bad, route.offsets, rows=route.rows)
    of_hit = hit[route.rows.long()]
    assert torch.equal(y.isnan(), of_hit[:, None].expand_as(y)) and torch.equal(y[~of_hit], rows[~of_hit])
    chosen = (r[1] == 2).any(dim=1)                           # the tokens of expert 2
    for which, column in ((0, None), (2, None), (4, 33)):
        W = [t.clone() for t in mlp]
        W[which][2, 33, 40] = 0x7f
        y = cuda_lib.qmm_f8_moe(x, route, *W)
        nan = torch.zeros_like(y, dtype=torch.bool)
        if column is None:
            nan[chosen] = True
        else:
            nan[chosen, column] = True
        assert torch.equal(y.isnan(), nan) and torch.equal(y[~nan], want[~nan])
    assert cuda_lib.qmm_device_status() == 0


# ---------------------------------------------------------------------------
# Copies that never come (the waits run out after about a second)
# ---------------------------------------------------------------------------
def _stalled(q, call, launches=1):
    import torch
    want = call()
    assert q.qmm_device_status() == 0
    q.inject_stall(launches)
    call()
    assert q.qmm_device_status() == q.QMM_ETIMEOUT
    assert q.qmm_device_status() == 0
    for _ in range(2):
        assert torch.equal(want, call())
    assert q.qmm_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(8, 1024, 5120), (300, 2000, 4096), (200, 10300, 9216), (1100, 14336, 1024)])
def test_stalled_copies_of_one_matrix(cuda_lib, M, N, K):
    """x quantised by the product; pairs of CTAs with tiles among several of them, shared by all, and whole ones."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    W, S = (t[0] for t in _matrices(g, 1, N, K, 1.0))
    x = _x(g, M, K)
    _stalled(cuda_lib, lambda: cuda_lib.qmm_f8(W, S, x))


@pytest.mark.parametrize("rows", [5, 100])
def test_stalled_copies_of_experts(cuda_lib, rows):
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    W, S = _matrices(g, 4, 1000, 2048, 1.0)
    x = _x(g, 4 * rows, 2048)
    offsets = torch.arange(5, dtype=torch.int32, device="cuda") * rows
    _stalled(cuda_lib, lambda: cuda_lib.qmm_f8_experts(W, S, x, offsets))


@pytest.mark.parametrize("T", [8, 100])
@pytest.mark.parametrize("launches", [1, 2])                  # gate and up; down as well
def test_stalled_copies_of_an_expert_layer(cuda_lib, T, launches):
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    *r, mlp = _layer(g, T, 2, 4, 1152, 1168)
    x = _x(g, T, 1152)
    route = _route(cuda_lib, *r)
    _stalled(cuda_lib, lambda: cuda_lib.qmm_f8_moe(x, route, *mlp), launches)

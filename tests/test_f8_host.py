"""Argument checks of the 8-bit-float entry points, before anything touches a GPU."""
import ctypes

import mat_mul_gb300 as q

NULL = ctypes.c_void_p(0)


def _buffer():
    buf = ctypes.create_string_buffer(8192)
    return buf, (ctypes.addressof(buf) + 15) & ~15


def test_product_refusals():
    L = q.load()
    buf, base = _buffer()
    P = ctypes.c_void_p

    def call(W=base, S=base, N=4, K=32, xt=0, x=base, M=2, ldx=32, yt=0, y=base, ldy=4):
        return L.qmm_f8(P(W), P(S), N, K, xt, P(x), M, ldx, yt, P(y), ldy, NULL)
    for kw in ({"xt": 3}, {"yt": -1}):
        assert call(**kw) == q.QMM_EINVAL_TYPE
    for kw in ({"K": 24}, {"K": -16}, {"N": -1}, {"M": -1}, {"K": (1 << 24) + 16}, {"N": 1 << 31}, {"M": 1 << 31},
               {"N": 1 << 30, "M": 1 << 30}, {"ldx": 31}, {"ldy": 3}):
        assert call(**kw) == q.QMM_EINVAL_SHAPE, kw
    for kw in ({"W": 0}, {"S": 0}, {"x": 0}, {"y": 0}, {"W": base + 8}, {"S": base + 2}, {"x": base + 1}, {"y": base + 2},
               {"xt": 1, "x": base + 1}, {"yt": 2, "y": base + 1}):
        assert call(**kw) == q.QMM_EINVAL_PTR, kw
    assert b"aligned" in L.qmm_last_error()
    before = L.qmm_launch_count()
    assert call(M=0) == q.QMM_OK and call(N=0) == q.QMM_OK
    assert L.qmm_last_error() == b"" and L.qmm_launch_count() == before


def test_quantize_refusals():
    L = q.load()
    buf, base = _buffer()
    P = ctypes.c_void_p
    assert L.qmm_f8_quantize(9, P(base), 1, 4, 4, P(base), P(base), NULL) == q.QMM_EINVAL_TYPE
    assert L.qmm_f8_quantize(0, P(base), -1, 4, 4, P(base), P(base), NULL) == q.QMM_EINVAL_SHAPE
    assert L.qmm_f8_quantize(0, P(base), 2, 4, 3, P(base), P(base), NULL) == q.QMM_EINVAL_SHAPE
    assert L.qmm_f8_quantize(0, NULL, 1, 4, 4, P(base), P(base), NULL) == q.QMM_EINVAL_PTR
    assert L.qmm_f8_quantize(0, P(base), 1, 4, 4, NULL, P(base), NULL) == q.QMM_EINVAL_PTR
    assert L.qmm_f8_quantize(0, P(base), 1, 4, 4, P(base), P(base + 2), NULL) == q.QMM_EINVAL_PTR
    assert L.qmm_f8_quantize(0, NULL, 0, 4, 4, NULL, NULL, NULL) == q.QMM_OK
    assert L.qmm_f8_quantize(0, NULL, 3, 0, 0, NULL, NULL, NULL) == q.QMM_OK


def test_experts_refusals():
    L = q.load()
    buf, base = _buffer()
    P = ctypes.c_void_p

    def call(W=base, E=2, N=4, K=32, M=3, off=base, rows=0, R=3, ldx=32, ldy=4, x=base):
        return L.qmm_f8_experts(P(W), P(base), E, N, K, 0, P(x), M, ldx, P(off), P(rows), R, 0, P(base), ldy, NULL)
    for kw in ({"E": 0}, {"E": q_max() + 1}, {"K": 8}, {"R": 4}, {"M": 2}, {"N": -4}, {"E": 1024, "N": 1 << 22},
               {"rows": base, "M": 0}, {"M": -1, "rows": base}, {"ldx": 16}, {"ldy": 1}):
        assert call(**kw) == q.QMM_EINVAL_SHAPE, kw
    for kw in ({"off": 0}, {"off": base + 2}, {"rows": base + 1}, {"W": base + 4}, {"x": 0}):
        assert call(**kw) == q.QMM_EINVAL_PTR, kw
    assert call(R=0, M=0, off=0) == q.QMM_OK


def q_max():
    return 1024


def test_route_refusals():
    L = q.load()
    buf, base = _buffer()
    P = ctypes.c_void_p

    def call(t=0, x=base, T=2, E=8, ldx=8, k=2, score=0, off=base, w=base, e=base, r=base, s=base):
        return L.qmm_route(t, P(x), T, E, ldx, k, score, 1, 1.0, P(w), P(e), P(off), P(r), P(s), NULL)
    for kw in ({"t": 5}, {"score": 2}):
        assert call(**kw) == q.QMM_EINVAL_TYPE, kw
    for kw in ({"k": 0}, {"k": 9}, {"E": 0}, {"E": 1025}, {"E": 64, "ldx": 64, "k": 33}, {"T": -1}, {"T": 1 << 30},
               {"ldx": 7}):
        assert call(**kw) == q.QMM_EINVAL_SHAPE, kw
    for kw in ({"x": 0}, {"off": 0}, {"w": 0}, {"e": base + 1}, {"r": 0}, {"s": 0}):
        assert call(**kw) == q.QMM_EINVAL_PTR, kw


def test_moe_refusals():
    L = q.load()
    buf, base = _buffer()
    P = ctypes.c_void_p

    def call(xt=0, x=base, T=2, H=32, ldx=32, k=2, w=base, off=base, sl=base, E=4, I=16, Wg=base, Sd=base, yt=0, y=base,
             ldy=32):
        return L.qmm_f8_moe(xt, P(x), T, H, ldx, k, P(w), P(off), P(sl), E, I, P(Wg), P(base), P(base), P(base), P(base),
                            P(Sd), yt, P(y), ldy, NULL)
    for kw in ({"xt": 4}, {"yt": 4}):
        assert call(**kw) == q.QMM_EINVAL_TYPE, kw
    for kw in ({"H": 24}, {"I": 8}, {"k": 5}, {"k": 0}, {"E": 0}, {"T": -1}, {"T": 1 << 30}, {"ldx": 31}, {"ldy": 31}):
        assert call(**kw) == q.QMM_EINVAL_SHAPE, kw
    for kw in ({"x": 0}, {"w": 0}, {"off": 0}, {"sl": base + 2}, {"Wg": base + 8}, {"Sd": 0}, {"y": 0}):
        assert call(**kw) == q.QMM_EINVAL_PTR, kw
    assert call(T=0, x=0, y=0) == q.QMM_OK


def test_status_name():
    assert q._strerror(q.QMM_EINDEX) == "QMM_EINDEX"

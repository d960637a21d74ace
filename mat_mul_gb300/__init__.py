"""Python binding of libqmm (include/qmm.h): argument marshalling only.

Every step of the computation runs in the CUDA kernels of libqmm.so; torch is
used for device memory and streams.  There is no CPU fallback: when the
library is missing or no GPU is present the calls raise.

    import mat_mul_gb300 as q
    y = q.qmm(q.Q4_K, W_blocks, N, K, x)          # x: cuda f32 [M, K] -> [M, N]
    ys = q.qmm_group([(q.Q4_K, Wg, N), (q.Q4_K, Wu, N)], K, x)   # one launch, shared x
    h = q.qmm_gate_up(q.Q4_K, Wg, q.Q4_K, Wu, N, K, x)           # silu(Wg x) * (Wu x)
    o = q.qmm_t(q.Q8_0, V_cache, H, T, D, p)      # p: [H, M, T] -> [H, M, D]
    w = q.qmm_dequant(q.Q6_K, blocks, n_elems)    # cuda f32 [n_elems]

A call runs on the current stream or on the one given as stream=, as if made
under torch.cuda.stream(stream): what it allocates belongs to that stream, and
the caller orders it after the work that makes its inputs and before the
work that reads its results.

Weights in 8-bit floats (e4m3 codes, one fp32 scale per 128 x 128 block), x and
y in float32, float16 or bfloat16:

    y = q.qmm_f8(W, S, x)                         # W [N, K] codes, S its scales, x [M, K] -> [M, N]
    r = q.qmm_route(logits, k)                    # a token's k experts, their weights, the pairs by expert
    y = q.qmm_f8_experts(W, S, x, r.offsets, rows=r.rows)   # W [E, N, K]: one row per (token, expert)
    y = q.qmm_f8_moe(x, r, Wg, Sg, Wu, Su, Wd, Sd)          # the whole gated expert MLP, [T, H]
    c, s = q.qmm_f8_quantize(x)                   # codes and scales of activations

The attention layer of a step, over a paged cache of 8-bit floats (e4m3 codes, one scale per page and head):

    rope = q.qmm_rope_table(128, base=500000.0, scaling="parts", scale=8.0, original=8192)
    cache = q.KvCache.empty(pages, heads, page=64, dim=128)
    x = q.qmm_rope(x, rope, positions)            # x [T, heads, dim]; inverse=True: its gradient
    qr = q.qmm_kv_append(cache, k, v, table, lengths, rope=rope, q=qh)   # k turned and stored, queries turned
    y = q.qmm_kv_attention(cache, qr, table, lengths)                    # [T, heads, dim]
"""
from __future__ import annotations

import collections
import ctypes
import functools
import math
import os
import struct

Q8_0, Q4_K, Q6_K, Q5_K, Q3_K, Q2_K = 0, 1, 2, 3, 4, 5  # Q5_K, Q3_K, Q2_K: qmm_dequant only so far
BLOCK_BYTES = {Q8_0: 34, Q4_K: 144, Q6_K: 210, Q5_K: 176, Q3_K: 110, Q2_K: 84}
BLOCK_WEIGHTS = {Q8_0: 32, Q4_K: 256, Q6_K: 256, Q5_K: 256, Q3_K: 256, Q2_K: 256}

QMM_OK = 0
QMM_EINVAL_TYPE = -1
QMM_EINVAL_SHAPE = -2
QMM_EINVAL_PTR = -3
QMM_ENOMEM = -4
QMM_ECUDA = -5
QMM_ETIMEOUT = -6
QMM_EINDEX = -7

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqmm.so")

_lib = None


class QmmError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_strerror(status)}: {detail}")


def build(force: bool = False) -> str:
    from . import buildlib
    return buildlib.build(force=force)


def load():
    """Load libqmm.so, (re)building it first when it is absent or older than
    its sources."""
    global _lib
    if _lib is not None:
        return _lib
    build()
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.qmm_dequant.argtypes = [I, P, I64, P]
    L.qmm.argtypes = [I, P, I64, I64, P, I64, P, P]
    L.qmm_noalloc.argtypes = [I, P, I64, I64, P, I64, P, P]
    L.qmm_quantize_act.argtypes = [P, I64, I64, P, P, P, P]
    L.qmm_group.argtypes = [I, P, P, P, I64, P, I64, P, P]
    L.qmm_t.argtypes = [I, P, I64, I64, I64, P, I64, P, P]
    L.qmm_gate_up.argtypes = [I, P, I, P, I64, I64, P, I64, P, P]
    L.qmm_strerror.argtypes = [I]
    L.qmm_strerror.restype = ctypes.c_char_p
    L.qmm_last_error.restype = ctypes.c_char_p
    L.qmm_device_status.argtypes = [P]
    L.qmm_launch_count.restype = I64
    L.qmm_set_decode_path.argtypes = [I]
    L.qmm_set_decode_path.restype = I
    L.qmm_set_prefill_path.argtypes = [I]
    L.qmm_set_prefill_path.restype = I
    L.qmm_inject_stall.argtypes = [I]
    L.qmm_inject_stall.restype = I
    L.qmm_f8_quantize.argtypes = [I, P, I64, I64, I64, P, P, P]
    L.qmm_f8.argtypes = [P, P, I64, I64, I, P, I64, I64, I, P, I64, P]
    L.qmm_f8_experts.argtypes = [P, P, I64, I64, I64, I, P, I64, I64, P, P, I64, I, P, I64, P]
    L.qmm_route.argtypes = [I, P, I64, I64, I64, I, I, I, ctypes.c_float, P, P, P, P, P, P]
    L.qmm_f8_moe.argtypes = [I, P, I64, I64, I64, I, P, P, P, I64, I64, P, P, P, P, P, P, I, P, I64, P]
    L.qmm_rope_turns.argtypes = [I, ctypes.c_double, P, I] + [ctypes.c_double] * 4 + [P]
    L.qmm_kv_attention_scratch.argtypes = [ctypes.c_char_p]
    L.qmm_kv_attention_scratch.restype = I64
    for f in ("qmm_rope", "qmm_kv_append", "qmm_kv_attention"):
        getattr(L, f).argtypes = [ctypes.c_char_p, P]  # the argument structure as packed bytes
        getattr(L, f).restype = I
    L.qmm_rope_turns.restype = I
    for f in ("qmm_f8_quantize", "qmm_f8", "qmm_f8_experts", "qmm_route", "qmm_f8_moe"):
        getattr(L, f).restype = I
    for f in ("qmm_dequant", "qmm", "qmm_noalloc", "qmm_quantize_act", "qmm_device_status",
              "qmm_release", "qmm_group", "qmm_t", "qmm_gate_up"):
        getattr(L, f).restype = I
    _lib = L
    return L


def _strerror(status: int) -> str:
    return load().qmm_strerror(int(status)).decode()


def _check(rc: int):
    if rc != QMM_OK:
        raise QmmError(rc, load().qmm_last_error().decode())


def _empty(shape, dtype, device, stream):
    """Memory for a result of a call on `stream` (None: the current one): from
    that stream's pool, since a block of the current stream's may still be in
    use there when the other stream writes it; and not handed out again before
    the current stream, where the caller reads it, is done with it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream.cuda_stream != here.cuda_stream:
        t.record_stream(here)
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


# The library works on the current device: its workspaces, its status word and
# its launches are there.  Tensors and streams of another one are refused.
_torch = None


def _current_device():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch._C._cuda_getDevice()  # (torch.cuda.current_device() without its look-ups: every call comes here)


def _refuse_device(t, current):
    raise ValueError(f"tensors on cuda:{t.get_device()}, but cuda:{current} is the current device: call under "
                     f"torch.cuda.device({t.get_device()})")


def _given_stream(stream, current):
    if getattr(stream, "device_index", current) != current:
        raise ValueError(f"a stream of cuda:{stream.device_index}, but cuda:{current} is the current device")
    return stream.cuda_stream


def _stream_handle(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(_given_stream(stream, _current_device()))


def _require_cuda(*ts):
    current = None
    for t in ts:
        if t is not None:
            d = t.get_device()
            if d != current:
                if d < 0:
                    raise ValueError("libqmm takes device tensors; got a tensor on " + str(t.device))
                if current is None:
                    current = _current_device()
                if d != current:
                    _refuse_device(t, current)


def qmm_dequant(qtype: int, blocks, n_elems: int, out=None):
    """Unpack n_elems weights of type qtype from a uint8 device tensor."""
    import torch
    _require_cuda(blocks, out)
    if out is None:
        out = _empty(n_elems, torch.float32, blocks.device, None)
    _check(load().qmm_dequant(int(qtype), _ptr(blocks), int(n_elems), _ptr(out)))
    return out


def qmm(qtype: int, W, N: int, K: int, x, y=None, stream=None):
    """y[M,N] = W . x^T for a uint8 device tensor W of packed blocks and a
    device f32 tensor x of shape [M, K] (or [K])."""
    import torch
    _require_cuda(W, x, y)
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    M = 1 if x.dim() == 1 else x.shape[0]
    if x.shape[-1] != K:
        raise ValueError(f"x has {x.shape[-1]} columns, K = {K}")
    if y is None:
        y = _empty((M, N), torch.float32, x.device, stream)
    elif y.dtype != torch.float32 or not y.is_contiguous() or y.device != x.device or y.numel() < M * N:
        raise ValueError(f"y must be a contiguous float32 tensor on {x.device} with at least M*N = {M * N} elements")
    _check(load().qmm(int(qtype), _ptr(W), int(N), int(K), _ptr(x), int(M), _ptr(y),
                      _stream_handle(stream)))
    return y


def qmm_t(qtype: int, W, H: int, N: int, K: int, x, y=None, stream=None):
    """y[h, m, k] = sum_n x[h, m, n] * w[h, n, k] for H matrices of N rows of
    K weights (uint8 device tensor W of packed Q8_0 blocks) and a device f32
    tensor x of shape [H, M, N]; returns y of shape [H, M, K]."""
    import torch
    _require_cuda(W, x, y)
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    if x.dim() != 3 or x.shape[0] != H or x.shape[2] != N:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [H={H}, M, N={N}]")
    M = x.shape[1]
    if y is None:
        y = _empty((H, M, K), torch.float32, x.device, stream)
    _check(load().qmm_t(int(qtype), _ptr(W), int(H), int(N), int(K), _ptr(x), int(M), _ptr(y),
                        _stream_handle(stream)))
    return y


def qmm_group(items, K: int, x, stream=None):
    """Several products that read the same x [M, K] (or [K]): items is a list
    of (qtype, W, N) or (qtype, W, N, y); returns the list of y tensors
    [M, N_i].  With M <= 8 the group is one decode launch."""
    import torch
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    M = 1 if x.dim() == 1 else x.shape[0]
    if x.shape[-1] != K:
        raise ValueError(f"x has {x.shape[-1]} columns, K = {K}")
    n = len(items)
    ys = []
    for it in items:
        y = it[3] if len(it) > 3 and it[3] is not None else _empty((M, int(it[2])), torch.float32, x.device, stream)
        _require_cuda(it[1], x, y)
        ys.append(y)
    types = (ctypes.c_int * max(n, 1))(*[int(it[0]) for it in items])
    Ws = (ctypes.c_void_p * max(n, 1))(*[_ptr(it[1]) for it in items])
    Ns = (ctypes.c_int64 * max(n, 1))(*[int(it[2]) for it in items])
    Ys = (ctypes.c_void_p * max(n, 1))(*[_ptr(y) for y in ys])
    _check(load().qmm_group(int(n), types, Ws, Ns, int(K), _ptr(x), int(M), Ys, _stream_handle(stream)))
    return ys


def qmm_gate_up(type_gate: int, W_gate, type_up: int, W_up, N: int, K: int, x, h=None, stream=None):
    """h[M,N] = silu(W_gate . x^T) * (W_up . x^T) for device x [M, K] (or
    [K]); one launch for M <= 2 when both matrices have one type."""
    import torch
    _require_cuda(W_gate, W_up, x, h)
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    M = 1 if x.dim() == 1 else x.shape[0]
    if x.shape[-1] != K:
        raise ValueError(f"x has {x.shape[-1]} columns, K = {K}")
    if h is None:
        h = _empty((M, N), torch.float32, x.device, stream)
    elif h.dtype != torch.float32 or not h.is_contiguous() or h.device != x.device or h.numel() < M * N:
        raise ValueError(f"h must be a contiguous float32 tensor on {x.device} with at least M*N = {M * N} elements")
    _check(load().qmm_gate_up(int(type_gate), _ptr(W_gate), int(type_up), _ptr(W_up), int(N), int(K), _ptr(x),
                              int(M), _ptr(h), _stream_handle(stream)))
    return h


def qmm_noalloc(qtype: int, W, N: int, K: int, x, y, stream=None):
    """Same product as qmm() without any device allocation by the library,
    for callers that keep all device memory in their own fixed pool or must
    not stall on cudaFree.  y [M, N] float32 must be given.  Uses a 16 MiB
    scratch inside the library image; calls that overlap on the GPU race on
    it."""
    import torch
    _require_cuda(W, x, y)
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    M = 1 if x.dim() == 1 else x.shape[0]
    if x.shape[-1] != K:
        raise ValueError(f"x has {x.shape[-1]} columns, K = {K}")
    if y.dtype != torch.float32 or not y.is_contiguous() or y.device != x.device or y.numel() < M * N:
        raise ValueError(f"y must be a contiguous float32 tensor on {x.device} with at least M*N = {M * N} elements")
    _check(load().qmm_noalloc(int(qtype), _ptr(W), int(N), int(K), _ptr(x), int(M), _ptr(y),
                              _stream_handle(stream)))
    return y


def qmm_quantize_act(x, stream=None):
    """Return (q int8 [M,K], d f32 [M,K/32], s int32 [M,K/32]) for device x."""
    import torch
    _require_cuda(x)
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    M, K = x2.shape
    q = _empty((M, K), torch.int8, x.device, stream)
    d = _empty((M, K // 32), torch.float32, x.device, stream)
    s = _empty((M, K // 32), torch.int32, x.device, stream)
    _check(load().qmm_quantize_act(_ptr(x2), int(M), int(K), _ptr(q), _ptr(d), _ptr(s),
                                   _stream_handle(stream)))
    return q, d, s


# ---------------------------------------------------------------------------
# Block-scaled 8-bit floats and expert layers
#
# A decode step makes these calls once per projection, with a few microseconds
# of GPU work each: the checks below read each tensor's attributes once, pass
# plain integers to the library and take the current stream's handle without
# making a stream object.
# ---------------------------------------------------------------------------
F8_BLOCK = 128          # values per scale along K, weight rows per scale along N
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1
_SCORES = {"softmax": ROUTE_SOFTMAX, "sigmoid": ROUTE_SIGMOID}
_f8 = None              # what the calls below need of torch and the library, made on first use


class _F8:
    def __init__(self):
        import torch
        self.lib = load()
        self.empty = torch.empty
        self.float32, self.int32, self.e4m3 = torch.float32, torch.int32, torch.float8_e4m3fn
        self.codes = (torch.float8_e4m3fn, torch.uint8)
        self.ftypes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # qmm_ftype
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
        self.current_device = torch._C._cuda_getDevice
        self.uint8 = torch.uint8
        self._capturing = torch.cuda.is_current_stream_capturing
        self._use = torch.cuda.stream

    def capturing(self, stream):
        """Whether a call on the stream goes into a graph."""
        if stream is None:
            return self._capturing()
        with self._use(stream):
            return self._capturing()

    def on(self, stream):
        """torch.empty on a call's stream."""
        return self.empty if stream is None else functools.partial(_empty, stream=stream)

    def ftype(self, dtype, what):
        t = self.ftypes.get(dtype)
        if t is None:
            raise ValueError(f"{what} must be float32, float16 or bfloat16, not {dtype}")
        return t


def _f8_state():
    global _f8
    if _f8 is None:
        _f8 = _F8()
    return _f8


def _device_index(f, first, *others):
    """The CUDA device of every tensor given (None: left out), the current one."""
    if not first.is_cuda:
        _require_cuda(first)
    dev = first.get_device()
    if dev != f.current_device():
        _refuse_device(first, f.current_device())
    for t in others:
        if t is not None and t.get_device() != dev:
            _require_cuda(t)
            raise ValueError(f"tensors on {first.device} and on {t.device}")
    return dev


def _rows2d(t, what):
    """t as rows of adjacent elements: (rows, columns, row pitch)."""
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        ld, one = t.stride()
        if one == 1 or cols <= 1:
            # (a pitch below the row length, as of an expanded tensor, is refused by the library)
            return rows, cols, ld if rows > 1 else cols
    elif len(shape) == 1 and (shape[0] <= 1 or t.stride(0) == 1):
        return 1, shape[0], shape[0]
    raise ValueError(f"{what} must be a matrix whose row elements are adjacent, got shape {tuple(shape)} "
                     f"strides {t.stride()}")


def _f8_weights(f, W, S, dims, what):
    """Shape of the codes W, after the checks of W and of its scales S."""
    shape = W.shape
    if W.dtype not in f.codes or len(shape) != dims or not W.is_contiguous():
        raise ValueError(f"{what}: codes must be a contiguous {dims}-d float8_e4m3fn (or uint8) tensor")
    want = (*shape[:-2], -(-shape[-2] // F8_BLOCK), -(-shape[-1] // F8_BLOCK))
    if S.dtype != f.float32 or S.shape != want or not S.is_contiguous():
        raise ValueError(f"{what}: scales must be a contiguous float32 tensor of shape {want}, got {tuple(S.shape)}")
    return shape


def _f8_out(f, y, rows, cols, dtype, device, stream):
    """The result tensor and its row pitch: y checked, or a new one."""
    if y is None:
        return f.on(stream)((rows, cols), dtype=dtype, device=device), cols
    r, c, ldy = _rows2d(y, "y")
    if r != rows or c != cols:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {(rows, cols)}")
    return y, ldy


def _int32(f, t, n, what):
    if t.dtype != f.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} elements, got {t.dtype} {tuple(t.shape)}")


def qmm_f8_quantize(x, stream=None):
    """(codes float8_e4m3fn [M, K], scales float32 [M, ceil(K/128)]) of a device
    tensor x [M, K] (or [K]) of float32, float16 or bfloat16 rows."""
    f = _f8_state()
    dev = _device_index(f, x)
    M, K, ldx = _rows2d(x, "x")
    ft = f.ftype(x.dtype, "x")
    device = x.device
    empty = f.on(stream)
    c = empty((M, K), dtype=f.e4m3, device=device)
    s = empty((M, -(-K // F8_BLOCK)), dtype=f.float32, device=device)
    rc = f.lib.qmm_f8_quantize(ft, x.data_ptr(), M, K, ldx, c.data_ptr(), s.data_ptr(),
                               f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return c, s


def qmm_f8(W, S, x, y=None, dtype=None, stream=None):
    """y[M, N] = W . x^T for codes W [N, K] (float8_e4m3fn or uint8), scales S
    [ceil(N/128), ceil(K/128)] and x [M, K] (or [K]) of float32, float16 or
    bfloat16; y has x's type unless dtype (or y) says otherwise.  K a multiple
    of 16.  Rows of x and y may be further apart than their length."""
    f = _f8_state()
    dev = _device_index(f, x, W, S, y)
    N, K = _f8_weights(f, W, S, 2, "W")
    M, cols, ldx = _rows2d(x, "x")
    if cols != K:
        raise ValueError(f"x has {cols} columns, W {K}")
    xt = x.dtype
    ft = f.ftype(xt, "x")
    y, ldy = _f8_out(f, y, M, N, dtype or xt, x.device, stream)
    rc = f.lib.qmm_f8(W.data_ptr(), S.data_ptr(), N, K, ft, x.data_ptr(), M, ldx, f.ftype(y.dtype, "y"), y.data_ptr(),
                      ldy, f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return y


def qmm_f8_experts(W, S, x, offsets, rows=None, y=None, dtype=None, stream=None):
    """The product grouped by expert: y[r] = W[e] . x[rows[r]] (or x[r] without
    rows) for offsets[e] <= r < offsets[e+1]; W [E, N, K] codes, S their scales,
    offsets int32 [E+1] and rows int32 on the device.  Returns y [R, N], R the
    length of rows (or of x); rows of y from offsets[E] on are not written."""
    f = _f8_state()
    dev = _device_index(f, x, W, S, offsets, rows, y)
    E, N, K = _f8_weights(f, W, S, 3, "W")
    M, cols, ldx = _rows2d(x, "x")
    if cols != K:
        raise ValueError(f"x has {cols} columns, W {K}")
    _int32(f, offsets, E + 1, "offsets")
    R, index = M, None
    if rows is not None:
        R = rows.numel()
        _int32(f, rows, R, "rows")
        index = rows.data_ptr()
    xt = x.dtype
    ft = f.ftype(xt, "x")
    y, ldy = _f8_out(f, y, R, N, dtype or xt, x.device, stream)
    rc = f.lib.qmm_f8_experts(W.data_ptr(), S.data_ptr(), E, N, K, ft, x.data_ptr(), M, ldx, offsets.data_ptr(), index, R,
                              f.ftype(y.dtype, "y"), y.data_ptr(), ldy,
                              f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return y


#: What qmm_route returns: weights [T, k] float32 and experts [T, k] int32 of each token's
#: choices, the groups offsets [E+1], the token of each sorted row rows [T*k], and the sorted
#: row of each pair slots [T, k] (all int32).
Route = collections.namedtuple("Route", "weights experts offsets rows slots")


def qmm_route(logits, k, score="softmax", normalize=True, factor=1.0, stream=None):
    """The k experts of each token with the largest logits [T, E], their weights
    (softmax or sigmoid scores, divided by their sum when normalize), and the
    (token, choice) pairs sorted by expert; see Route."""
    f = _f8_state()
    dev = _device_index(f, logits)
    T, E, ld = _rows2d(logits, "logits")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    k = int(k)
    n = k if k > 0 else 0
    ft, device, empty, i32 = f.ftype(logits.dtype, "logits"), logits.device, f.on(stream), f.int32
    weights = empty((T, n), dtype=f.float32, device=device)
    # (five allocations: views of one buffer cost more than twice as much)
    experts = empty((T, n), dtype=i32, device=device)
    slots = empty((T, n), dtype=i32, device=device)
    rows = empty(T * n, dtype=i32, device=device)
    offsets = empty(E + 1, dtype=i32, device=device)
    rc = f.lib.qmm_route(ft, logits.data_ptr(), T, E, ld, k, _SCORES[score], 1 if normalize else 0, factor,
                         weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(),
                         f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return Route(weights, experts, offsets, rows, slots)


def qmm_f8_moe(x, route, W_gate, S_gate, W_up, S_up, W_down, S_down, y=None, dtype=None, stream=None):
    """y[t] = sum_j weights[t, j] * W_down[e] . h, h = silu(W_gate[e] . x[t]) *
    (W_up[e] . x[t]), over the choices of route (a Route, as qmm_route returns
    it): x [T, H], W_gate and W_up [E, I, H], W_down [E, H, I] codes with their
    scales.  H and I multiples of 16."""
    f = _f8_state()
    weights, _, offsets, _, slots = route
    dev = _device_index(f, x, W_gate, S_gate, W_up, S_up, W_down, S_down, weights, offsets, slots, y)
    E, I, H = shape = _f8_weights(f, W_gate, S_gate, 3, "W_gate")
    if _f8_weights(f, W_up, S_up, 3, "W_up") != shape or _f8_weights(f, W_down, S_down, 3, "W_down") != (E, H, I):
        raise ValueError(f"W_up must be {(E, I, H)} and W_down {(E, H, I)} for W_gate {(E, I, H)}, got "
                         f"{tuple(W_up.shape)} and {tuple(W_down.shape)}")
    T, cols, ldx = _rows2d(x, "x")
    if cols != H:
        raise ValueError(f"x has {cols} columns, the experts {H}")
    wshape = weights.shape
    if len(wshape) != 2 or wshape[0] != T or weights.dtype != f.float32 or not weights.is_contiguous():
        raise ValueError(f"route.weights must be a contiguous float32 tensor of {T} rows, got {tuple(wshape)}")
    k = wshape[1]
    _int32(f, offsets, E + 1, "route.offsets")
    _int32(f, slots, T * k, "route.slots")
    xt = x.dtype
    ft = f.ftype(xt, "x")
    y, ldy = _f8_out(f, y, T, H, dtype or xt, x.device, stream)
    rc = f.lib.qmm_f8_moe(ft, x.data_ptr(), T, H, ldx, k, weights.data_ptr(), offsets.data_ptr(), slots.data_ptr(), E, I,
                          W_gate.data_ptr(), S_gate.data_ptr(), W_up.data_ptr(), S_up.data_ptr(), W_down.data_ptr(),
                          S_down.data_ptr(), f.ftype(y.dtype, "y"), y.data_ptr(), ldy,
                          f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return y


# ---------------------------------------------------------------------------
# The attention layer: position rotation, a paged cache of 8-bit floats, and
# attention over it.  The C calls take a structure of 64-bit fields, packed here
# in one go: a ctypes call with twenty arguments costs more than the kernel of a
# decode step.
# ---------------------------------------------------------------------------
_ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "parts": 3, "yarn": 3}
_ROPE_ARGS = struct.Struct("=QqQqqqqQqqqQqq")
_APPEND_ARGS = struct.Struct("=QQqqQQqqqQqqQqqQQQqqqQqq")
_ATTENTION_ARGS = struct.Struct("=QQqqQQqqqQqqqqQqqdqqQQq")


class _CacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
               [(n, ctypes.c_int64) for n in ("pages", "heads", "page", "dim")]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int64), ("interleaved", ctypes.c_int64),
                ("factor", ctypes.c_double)]


class RopeTable:
    """A rotation as qmm_rope_table makes it: turns (int64 [rot / 2], 2^64ths of a
    full turn per position), rot, interleaved, factor."""
    __slots__ = ("_turns", "_struct", "_at", "_device")

    def __init__(self, turns, rot, interleaved=False, factor=1.0):
        import torch
        _require_cuda(turns)
        if turns.dtype != torch.int64 or tuple(turns.shape) != (rot // 2,) or not turns.is_contiguous():
            raise ValueError(f"turns must be a contiguous int64 tensor of {rot // 2} elements, got {turns.dtype} "
                             f"{tuple(turns.shape)}")
        self._turns, self._device = turns, turns.get_device()
        self._struct = _RopeStruct(turns.data_ptr(), rot, 1 if interleaved else 0, factor)
        self._at = ctypes.addressof(self._struct)

    turns = property(lambda self: self._turns)
    rot = property(lambda self: self._struct.rot)
    interleaved = property(lambda self: bool(self._struct.interleaved))
    factor = property(lambda self: self._struct.factor)


def qmm_rope_table(rot, base=10000.0, interleaved=False, scaling=None, scale=1.0, original=None, low=None, high=None,
                   freqs=None, factor=None, device=None):
    """The rotation of the first rot values of a head: pairs (i, i + rot/2), or
    (2i, 2i + 1) when interleaved, at base^(-2i/rot) radians per position (or
    freqs[i]).  scaling: None, "linear" (positions divided by scale), "ntk" (a
    larger base), "parts" (frequencies with fewer than `low` turns within the
    `original` length divided by scale, those with more than `high` kept, 1 and
    4 unless given) or "yarn" (the same with 1 and 32, and the factor 0.1
    ln(scale) + 1).  factor multiplies the rotated values.

    "yarn" blends as the paper's text says, linear in the turns.  Many published
    checkpoints were tuned with a blend linear in the pair's index; theirs are
    freqs=[f * k + f / scale * (1 - k)] with f = base^(-2i/rot), 1 - k =
    (i - i(high)) / (i(low) - i(high)) within 0 .. 1 and i(r) = rot / 2 *
    log(original / (2 pi r)) / log(base), and factor=0.1 ln(scale) + 1; some
    round i(high) down and i(low) up."""
    import torch
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be None, 'linear', 'ntk', 'parts' or 'yarn', not {scaling!r}")
    if scaling in ("parts", "yarn") and original is None:
        raise ValueError(f"scaling {scaling!r} needs the original length")
    rot = int(rot)
    n = max(rot // 2, 0)
    if freqs is not None:
        freqs = [float(f) for f in freqs]
        if len(freqs) != n:
            raise ValueError(f"{len(freqs)} frequencies for {n} pairs")
        freqs = (ctypes.c_double * max(n, 1))(*freqs)
    if factor is None:
        factor = 0.1 * math.log(scale) + 1.0 if scaling == "yarn" and scale > 1.0 else 1.0
    turns = (ctypes.c_uint64 * max(n, 1))()
    _check(load().qmm_rope_turns(rot, float(base), freqs, _ROPE_SCALINGS[scaling], float(scale), float(original or 0.0),
                                 float(1.0 if low is None else low),
                                 float((32.0 if scaling == "yarn" else 4.0) if high is None else high), turns))
    t = torch.frombuffer(bytearray(bytes(turns)[:8 * n]), dtype=torch.int64) if n else torch.empty(0, dtype=torch.int64)
    return RopeTable(t.to("cuda" if device is None else device), rot, interleaved, factor)


class KvCache:
    """The cache of one layer: k and v codes (float8_e4m3fn or uint8 [pages,
    heads, page, dim]) and their scales (float32 [pages, heads]), tensors of the
    caller that the calls write to."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "heads", "page", "dim", "_struct", "_at", "_device", "_frozen")

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        _require_cuda(k, v, k_scale, v_scale)
        shape = tuple(k.shape)
        for t in (k, v):
            if t.dtype not in (torch.float8_e4m3fn, torch.uint8) or tuple(t.shape) != shape or len(shape) != 4 or \
                    not t.is_contiguous():
                raise ValueError("k and v must be contiguous float8_e4m3fn (or uint8) tensors of one shape [pages, heads, "
                                 f"page, dim], got {tuple(k.shape)} and {tuple(v.shape)}")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or tuple(t.shape) != shape[:2] or not t.is_contiguous():
                raise ValueError(f"scales must be contiguous float32 tensors of shape {shape[:2]}, got {tuple(t.shape)}")
        if shape[2] not in (16, 32, 64, 128) or shape[3] % 16 or not 16 <= shape[3] <= 256:
            raise ValueError(f"pages of 16, 32, 64 or 128 tokens, heads of a multiple of 16 up to 256 values, got {shape}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.heads, self.page, self.dim = shape[1:]
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *shape)
        self._at, self._device = ctypes.addressof(self._struct), k.get_device()
        self._frozen = True

    def __setattr__(self, name, value):
        # (the calls use the addresses of the tensors that the cache was made of)
        if getattr(self, "_frozen", False):
            raise AttributeError("a cache keeps its tensors; make another one")
        object.__setattr__(self, name, value)

    @classmethod
    def empty(cls, pages, heads, page=64, dim=128, device=None):
        """A cache of zeros."""
        import torch
        device = "cuda" if device is None else device
        k, v = (torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                for _ in range(2))
        ks, vs = (torch.zeros((pages, heads), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _row_heads(t, what):
    """t [T, heads, dim] with adjacent elements of a head: (T, heads, dim, pitch
    of rows, pitch of heads)."""
    if t.dim() == 3:
        T, H, D = t.shape
        a, b, one = t.stride()
        if one == 1 or D <= 1:
            return T, H, D, a, b
    raise ValueError(f"{what} must be [rows, heads, dim] with the elements of a head adjacent, got shape "
                     f"{tuple(t.shape)} strides {t.stride()}")


def _row_heads_out(f, y, T, H, D, dtype, like, stream, what):
    if y is None:
        return f.on(stream)((T, H, D), dtype=dtype, device=like.device), H * D, D
    r, h, d, a, b = _row_heads(y, what)
    if (r, h, d) != (T, H, D):
        raise ValueError(f"{what} has shape {tuple(y.shape)}, expected {(T, H, D)}")
    return y, a, b


def _kv_batch(f, cache, T, table, lengths, offsets):
    """(sequences, table width, its row pitch, address of the offsets) after the checks of a batch."""
    shape = table.shape
    if table.dtype != f.int32 or len(shape) != 2:
        raise ValueError(f"table must be an int32 matrix [sequences, pages], got {table.dtype} {tuple(shape)}")
    B, width = shape
    ld, one = table.stride()
    if one != 1 and width > 1:
        raise ValueError("the entries of a row of table must be adjacent")
    _int32(f, lengths, B, "lengths")
    if offsets is None:
        if T != B:
            raise ValueError(f"{T} rows of {B} sequences: without offsets every sequence has one row")
        return B, width, ld, 0
    _int32(f, offsets, B + 1, "offsets")
    return B, width, ld, offsets.data_ptr()


def _kv_device(f, cache, rope, first, *others):
    dev = _device_index(f, first, *others)
    if cache is not None and cache._device != dev:
        raise ValueError(f"a cache on cuda:{cache._device}, rows on {first.device}")
    if rope is not None and rope._device != dev:
        raise ValueError(f"a rotation table on cuda:{rope._device}, rows on {first.device}")
    return dev


def qmm_rope(x, rope, positions, y=None, inverse=False, dtype=None, stream=None):
    """The heads of x [T, heads, dim] turned by rope (a RopeTable) at positions
    (int32 [T]); with inverse by the negative angles, which is the gradient.  y:
    the result, which may be x."""
    f = _f8_state()
    dev = _kv_device(f, None, rope, x, positions, y)
    T, H, D, a, b = _row_heads(x, "x")
    _int32(f, positions, T, "positions")
    xt = x.dtype
    ft = f.ftype(xt, "x")
    y, c, d = _row_heads_out(f, y, T, H, D, dtype or xt, x, stream, "y")
    rc = f.lib.qmm_rope(_ROPE_ARGS.pack(rope._at, 1 if inverse else 0, positions.data_ptr(), T, H, D, ft, x.data_ptr(), a, b,
                                        f.ftype(y.dtype, "y"), y.data_ptr(), c, d),
                        f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return y


def qmm_kv_append(cache, k, v, table, lengths, offsets=None, rope=None, positions=None, q=None, q_out=None, stream=None):
    """The new keys and values k, v [T, heads, dim] into the cache (a KvCache), the
    keys turned by rope on the way; with q [T, query heads, dim] returns the
    queries turned too (q_out may be q), else None.  Rows offsets[b] ..
    offsets[b+1] (int32 [B+1]; row b without offsets) are the last of the
    lengths[b] tokens of sequence b, token j of which is in page table[b, j //
    page]; table int32 [B, width], lengths int32 [B].  positions int32 [T]: other
    angles than those of a row's place in its sequence."""
    f = _f8_state()
    dev = _kv_device(f, cache, rope, k, v, table, lengths, offsets, positions, q, q_out)
    T, H, D, a, b = _row_heads(k, "k")
    r, h, d, vc, vd = _row_heads(v, "v")
    if H != cache.heads or D != cache.dim or (r, h, d) != (T, H, D):
        raise ValueError(f"k and v must be {(T, cache.heads, cache.dim)}, got {tuple(k.shape)} and {tuple(v.shape)}")
    xt = k.dtype
    ft = f.ftype(xt, "k")
    if v.dtype != xt:
        raise ValueError(f"k is {xt}, v {v.dtype}")
    B, width, ld, off = _kv_batch(f, cache, T, table, lengths, offsets)
    if positions is not None:
        _int32(f, positions, T, "positions")
    qp = Hq = qa = qb = op = oa = ob = 0
    if q is not None:
        r, Hq, d, qa, qb = _row_heads(q, "q")
        if (r, d) != (T, D) or q.dtype != xt:
            raise ValueError(f"q must be [{T}, query heads, {D}] of {xt}, got {tuple(q.shape)} of {q.dtype}")
        if rope is None:
            raise ValueError("queries are only turned: q needs rope")
        qp = q.data_ptr()
        q_out, oa, ob = _row_heads_out(f, q_out, T, Hq, D, xt, q, stream, "q_out")
        if q_out.dtype != xt:
            raise ValueError(f"q_out is {q_out.dtype}, q {xt}")
        op = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = f.lib.qmm_kv_append(_APPEND_ARGS.pack(cache._at, table.data_ptr(), width, ld, lengths.data_ptr(), off, B, T, ft,
                                               k.data_ptr(), a, b, v.data_ptr(), vc, vd, 0 if rope is None else rope._at,
                                               0 if positions is None else positions.data_ptr(), qp, Hq, qa, qb, op, oa, ob),
                             f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return q_out


def qmm_kv_attention(cache, q, table, lengths, offsets=None, scale=None, causal=True, window=0, y=None, dtype=None,
                     lse=False, stream=None):
    """softmax(scale * q k^T) v of the rows q [T, query heads, dim] over the tokens
    of their sequences in the cache (a KvCache); table, lengths and offsets as in
    qmm_kv_append, scale 1/sqrt(dim) unless given.  A causal row sees the tokens
    up to its own (the last `window` of them if that is not 0); a row that sees
    none gets 0.  Returns y [T, query heads, dim], with lse also the log of the
    sum of the exponentials, float32 [T, query heads].  Rows from offsets[-1] on
    are not written."""
    f = _f8_state()
    dev = _kv_device(f, cache, None, q, table, lengths, offsets, y)
    T, H, D, a, b = _row_heads(q, "q")
    if D != cache.dim:
        raise ValueError(f"q has heads of {D} values, the cache of {cache.dim}")
    B, width, ld, off = _kv_batch(f, cache, T, table, lengths, offsets)
    qt = q.dtype
    ft = f.ftype(qt, "q")
    y, c, d = _row_heads_out(f, y, T, H, D, dtype or qt, q, stream, "y")
    sums = f.on(stream)((T, H), dtype=f.float32, device=q.device) if lse else None
    head = (cache._at, table.data_ptr(), width, ld, lengths.data_ptr(), off, B, T, ft, q.data_ptr(), H, a, b,
            f.ftype(y.dtype, "y"), y.data_ptr(), c, d, 1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0, window,
            sums.data_ptr() if lse else 0)
    if f.capturing(stream):
        # a graph has its partial results in its own memory, so that two of one stream can run at once
        n = f.lib.qmm_kv_attention_scratch(_ATTENTION_ARGS.pack(*head, 0, 0))
        if n < 0:
            _check(int(n))
        work = f.on(stream)(n, dtype=f.uint8, device=q.device)
        args = _ATTENTION_ARGS.pack(*head, work.data_ptr(), n)
    else:
        args = _ATTENTION_ARGS.pack(*head, 0, 0)
    rc = f.lib.qmm_kv_attention(args, f.stream(dev) if stream is None else _given_stream(stream, dev))
    if rc:
        _check(rc)
    return (y, sums) if lse else y


def qmm_device_status(stream=None) -> int:
    return int(load().qmm_device_status(_stream_handle(stream)))


def qmm_release() -> None:
    _check(load().qmm_release())


def qmm_launch_count() -> int:
    return int(load().qmm_launch_count())


# Decode kernel choice (qmm_set_decode_path in the C header).
DECODE_AUTO, DECODE_BLOCK, DECODE_TENSOR, DECODE_ROWS = 0, 1, 2, 3


def set_decode_path(path: int) -> int:
    """Select the decode kernel for every later call; returns the previous path."""
    rc = int(load().qmm_set_decode_path(int(path)))
    if rc < 0:
        raise QmmError(rc, load().qmm_last_error().decode())
    return rc


# Prefill kernel choice (qmm_set_prefill_path in the C header).
PREFILL_AUTO, PREFILL_INT8 = 0, 1


def set_prefill_path(path: int) -> int:
    """Select the prefill kernel for every later call; returns the previous path."""
    rc = int(load().qmm_set_prefill_path(int(path)))
    if rc < 0:
        raise QmmError(rc, load().qmm_last_error().decode())
    return rc


def inject_stall(launches: int) -> int:
    """Failure-detection test hook: the next `launches` weight-streaming
    launches stop their first CTA's copies after one stage, so a bounded wait
    expires and qmm_device_status() reports QMM_ETIMEOUT.  Returns the
    previous pending count."""
    rc = int(load().qmm_inject_stall(int(launches)))
    if rc < 0:
        raise QmmError(rc, load().qmm_last_error().decode())
    return rc

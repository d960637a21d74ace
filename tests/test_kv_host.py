"""The position rotation, the paged cache and the attention over it, host side: what is refused before anything is
launched, the kernels that calls reach, their memory.  On the CPU."""
import ctypes

import pytest

import mat_mul_gb300 as q
from host_calls import run

MORE = """
def cache(pages=100, heads=4, page=64, dim=128, k=A, v=A, ks=A, vs=A):
    return q._CacheStruct(k, v, ks, vs, pages, heads, page, dim)
KEEP = []
def at(s):
    KEEP.append(s)
    return ctypes.addressof(s) if s is not None else 0
def table(rot=128, turns=A, inter=0, factor=1.0):
    return q._RopeStruct(turns, rot, inter, factor)
def rope(T=3, heads=4, dim=128, r=table(), inverse=0, pos=A, xt=2, x=A, xa=512, xb=128, yt=2, y=A + (1 << 20), ya=512, yb=128):
    return L.qmm_rope(q._ROPE_ARGS.pack(at(r), inverse, pos, T, heads, dim, xt, x, xa, xb, yt, y, ya, yb), ST)
def append(c=cache(), tab=A, width=8, ld=8, lens=A, off=0, B=3, T=3, t=2, k=A, ka=512, kb=128, v=A, va=512, vb=128, r=table(),
           pos=0, qp=A, Hq=8, qa=1024, qb=128, op=A + (1 << 20), oa=1024, ob=128):
    return L.qmm_kv_append(q._APPEND_ARGS.pack(at(c), tab, width, ld, lens, off, B, T, t, k, ka, kb, v, va, vb, at(r), pos, qp, Hq,
                                               qa, qb, op, oa, ob), ST)
def args(c=cache(), tab=A, width=8, ld=8, lens=A, off=0, B=3, T=3, t=2, x=A, Hq=8, xa=1024, xb=128, yt=2, y=A + 4096, ya=1024, yb=128,
         scale=0.1, causal=1, window=0, lse=0, work=0, n=0):
    return q._ATTENTION_ARGS.pack(at(c), tab, width, ld, lens, off, B, T, t, x, Hq, xa, xb, yt, y, ya, yb, scale, causal, window,
                                  lse, work, n)
def attend(**k): return L.qmm_kv_attention(args(**k), ST)
TYPE, SHAPE, PTR = q.QMM_EINVAL_TYPE, q.QMM_EINVAL_SHAPE, q.QMM_EINVAL_PTR
"""


def test_refusals(tmp_path):
    run(tmp_path, MORE + """
log()
def refused(call, code, *cases):
    for kw in cases:
        assert call(**kw) == code, (kw, L.qmm_last_error())
        assert L.qmm_last_error() != b''
I31 = 1 << 31
refused(rope, TYPE, dict(xt=3), dict(yt=-1), dict(xt=1 << 32))
refused(rope, SHAPE, dict(T=-1), dict(T=I31), dict(heads=-1), dict(heads=1 << 17), dict(dim=127), dict(dim=1 << 17), dict(r=table(130)),
        dict(r=table(3)), dict(r=table(-2)), dict(yb=127), dict(ya=511), dict(ya=0), dict(yb=0), dict(y=A, ya=1024),
        dict(y=A, yt=0, x=A, xt=1), dict(T=1 << 30, heads=4))
refused(rope, PTR, dict(r=None), dict(pos=0), dict(pos=A + 2), dict(x=0), dict(y=0), dict(x=A + 1), dict(y=A + 1), dict(r=table(turns=0)),
        dict(r=table(turns=A + 4)), dict(xt=0, x=A + 2))
refused(append, TYPE, dict(t=3), dict(t=-1))
for call in (append, attend):
    refused(call, SHAPE, dict(c=cache(heads=0)), dict(c=cache(heads=2000)), dict(c=cache(page=48)), dict(c=cache(page=256)), dict(c=cache(dim=8)),
            dict(c=cache(dim=272)), dict(c=cache(dim=100)), dict(c=cache(pages=-1)), dict(c=cache(pages=I31)), dict(c=cache(pages=0)),
            dict(T=-1), dict(B=-1), dict(B=4), dict(T=2), dict(width=-1), dict(width=1 << 26), dict(ld=7))
    refused(call, PTR, dict(c=None), dict(c=cache(k=0)), dict(c=cache(v=A + 8)), dict(c=cache(ks=0)), dict(c=cache(vs=A + 2)), dict(lens=0),
            dict(lens=A + 1), dict(off=A + 2, T=9), dict(tab=0), dict(tab=A + 2))
refused(append, SHAPE, dict(r=table(130)), dict(Hq=0), dict(Hq=1 << 15), dict(oa=1023), dict(ob=100), dict(op=A, oa=2048))
refused(append, PTR, dict(k=0), dict(v=0), dict(k=A + 1), dict(qp=A + 1), dict(op=0), dict(op=A + 1), dict(r=None), dict(pos=A + 1))
refused(attend, TYPE, dict(t=3), dict(yt=7))
refused(attend, SHAPE, dict(Hq=6), dict(Hq=0), dict(Hq=1 << 15), dict(window=-1), dict(window=5, causal=0), dict(scale=float('nan')),
        dict(scale=float('inf')), dict(scale=1e31), dict(ya=1023), dict(yb=64), dict(T=1 << 30, off=A, B=1),
        dict(work=A, n=100), dict(work=A, n=-1))
refused(attend, PTR, dict(x=0), dict(y=0), dict(x=A + 1), dict(y=A + 1), dict(lse=A + 2), dict(work=A + 128, n=1 << 30), dict(x=A, y=A))
refused(attend, SHAPE, dict(c=cache(pages=I31 >> 10, heads=1024), Hq=1024, xa=1 << 17, ya=1 << 17))
assert L.qmm_rope(None, ST) == PTR and L.qmm_kv_append(None, ST) == PTR and L.qmm_kv_attention(None, ST) == PTR
assert L.qmm_kv_attention_scratch(None) == PTR and L.qmm_kv_attention_scratch(args(Hq=6)) == SHAPE
assert not log('launch')
# nothing to do
for rc in (rope(T=0, x=0, y=0, pos=0), rope(heads=0), rope(dim=0, r=table(0)), append(B=0, T=0, k=0), append(T=0, off=A), attend(B=0, T=0, x=0, y=0),
           attend(T=0, off=A), attend(c=cache(pages=0), B=0, T=0)):
    assert rc == 0 and L.qmm_last_error() == b''
assert L.qmm_kv_attention_scratch(args(B=0, T=0)) == 0
assert not log('launch')
# and what is at the edge of it
for rc in (rope(r=table(0)), rope(x=A, y=A), rope(ya=128, yb=128 * 3, xa=128, xb=384), append(r=None, qp=0, op=0), append(r=table(0)), append(qp=A, op=A),
           append(qp=0), attend(window=1 << 40), attend(causal=0), attend(width=0, tab=0), attend(scale=0.0), attend(scale=-1.0),
           attend(c=cache(pages=(I31 >> 10) - 1, heads=1024), Hq=1024, xa=1 << 17, ya=1 << 17)):
    assert rc == 0, L.qmm_last_error()
assert len(log('launch')) == 13
""")


def test_table_refusals_and_values():
    L = q.load()
    t = (ctypes.c_uint64 * 8)()
    f = (ctypes.c_double * 8)(*[float("inf")] * 8)

    def call(rot=16, base=10000.0, freqs=None, scaling=0, scale=2.0, original=100.0, low=1.0, high=4.0, turns=t):
        return L.qmm_rope_turns(rot, base, freqs, scaling, scale, original, low, high, turns)
    for kw in (dict(rot=-2), dict(rot=3), dict(base=0.0), dict(base=float("inf")), dict(scaling=1, scale=0.0), dict(scaling=2, rot=2),
               dict(scaling=2, freqs=f), dict(scaling=3, original=0.0), dict(scaling=3, low=4.0), dict(freqs=f), dict(base=float("nan"))):
        assert call(**kw) == q.QMM_EINVAL_SHAPE, kw
    assert call(scaling=4) == q.QMM_EINVAL_TYPE and call(scaling=-1) == q.QMM_EINVAL_TYPE
    assert call(turns=None) == q.QMM_EINVAL_PTR
    assert call() == 0 and call(rot=0, turns=None) == 0
    # a whole number of turns per position is none, a quarter is 2^62
    import math
    g = (ctypes.c_double * 4)(0.0, 2 * math.pi, math.pi / 2, -math.pi / 2)
    assert call(rot=8, freqs=g) == 0
    assert list(t)[:4] == [0, 0, 1 << 62, 3 << 62]


def test_no_kernel_is_out_of_reach(tmp_path):
    run(tmp_path, MORE + """
for xt in range(3):
    for yt in range(3):
        for dim, r in ((128, table(128)), (128, table(8)), (66, table(6)), (80, table(40))):
            assert rope(dim=dim, xb=dim, xa=4 * dim, yb=dim, ya=4 * dim, r=r, xt=xt, yt=yt) == 0
    for page, dim in ((64, 128), (128, 128), (128, 256), (16, 80)):
        for rot in (dim, 8, 6):
            for off, T in ((0, 3), (A, 9)):
                for qp in (0, A):
                    assert append(c=cache(page=page, dim=dim), t=xt, off=off, T=T, r=table(rot), qp=qp, kb=dim, vb=dim, qb=dim, ob=dim, oa=8 * dim) == 0
    for dim in (48, 64, 96, 128, 144, 256):
        for T in (3, 18, 45, 200):
            for width in (8, 400):
                assert attend(c=cache(dim=dim), t=xt, off=A, T=T, xb=dim, yb=dim, Hq=4 if T == 3 else 8, xa=2048, ya=2048, width=width, ld=width) == 0
launched = {e[2] for e in log('launch')}
mine = {k for k in kernels() if 'kv_' in k or 'rope_' in k}
assert len(mine) > 50 and launched <= set(kernels())
assert mine == launched, sorted(mine - launched)
""")


def test_rows_go_to_the_other_kernel_where_the_compiler_gave_too_few_registers(tmp_path):
    run(tmp_path, MORE + """
def names(n):
    log()
    fake.fake_registers(n)
    assert attend(off=A, T=600) == 0 and attend(off=A, T=600, t=0) == 0, L.qmm_last_error()
    return [e[2] for e in log('launch')]
fake.fake_registers(64)
assert attend(off=A, T=18, width=400, ld=400) == 0 and 'kv_attention_kernel' in log('launch')[-1][2]
fake.fake_registers(168)
assert attend(off=A, T=18, width=400, ld=400) == 0 and 'kv_attention_slim' in log('launch')[-1][2]
assert all('kv_attention_kernel' in n for n in names(64))
assert 'kv_attention_tc' in names(80)[0] and 'kv_attention_kernel' in names(80)[1]
for n in (0, 168):
    assert 'kv_attention_tc' in names(n)[0] and 'kv_attention_rows' in names(n)[1]
""")


def test_memory(tmp_path):
    """The stream's workspace and counters, allocated once; none of them where the caller gives scratch, whose counters
    are cleared by each call; a refused allocation leaves no error behind."""
    run(tmp_path, MORE + """
for kw in (dict(), dict(off=A, T=600)):
    assert L.qmm_release() == 0
    log()
    n = L.qmm_kv_attention_scratch(args(**kw))
    assert n > 0 and attend(work=A, n=n, **kw) == 0 and attend(work=A, n=n - 256, **kw) == SHAPE
    e = log()
    assert not [x for x in e if x[1] == 'malloc' and x[4] > 256], e
    clear = [x for x in e if x[1] == 'memset-async']
    assert len(clear) == 1 and A <= clear[0][3] and clear[0][3] + clear[0][4] <= A + n, (clear, n)
    assert attend(**kw) == 0 and attend(**kw) == 0
    assert len([x for x in log() if x[1] == 'malloc']) == 2
    assert L.qmm_release() == 0
    settle(most=1 << 12)
    assert attend(**kw) == q.QMM_ENOMEM
    settle()
    assert fake.fake_last_error() == 0
    assert attend(**kw) == 0
""")


# ---------------------------------------------------------------------------
# the Python binding
# ---------------------------------------------------------------------------
torch = pytest.importorskip("torch")
import binding  # noqa: E402


def _calls(index=0, other=None):
    """(name, call(stream)) on tensors of device `index`; the tensor named `other` is on the next one."""
    def t(name, *shape, dtype=torch.bfloat16):
        return binding.on_gpu(torch.zeros(shape, dtype=dtype), index + (name == other))
    i32, f8 = torch.int32, torch.float8_e4m3fn

    def cache():
        c = q.KvCache.__new__(q.KvCache)
        for n, v in (("k", None), ("heads", 2), ("page", 16), ("dim", 32), ("_at", 0x1000), ("_device", index + (other == "cache"))):
            object.__setattr__(c, n, v)
        return c

    def rope():
        r = q.RopeTable.__new__(q.RopeTable)
        r._at, r._device = 0x2000, index + (other == "rope")
        return r
    tab, lens = t("table", 3, 4, dtype=i32), t("lengths", 3, dtype=i32)
    return {
        "qmm_rope": lambda s: q.qmm_rope(t("x", 3, 4, 32), rope(), t("positions", 3, dtype=i32), stream=s),
        "qmm_kv_append": lambda s: q.qmm_kv_append(cache(), t("k", 3, 2, 32), t("v", 3, 2, 32), tab, lens, rope=rope(),
                                                   q=t("q", 3, 4, 32), stream=s),
        "qmm_kv_attention": lambda s: q.qmm_kv_attention(cache(), t("x", 3, 4, 32), tab, lens, lse=True, stream=s),
    }


@pytest.fixture
def lib(monkeypatch):
    with binding.stand_in(monkeypatch) as (lib, allocated):
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        yield lib, allocated


NAMES = ["qmm_rope", "qmm_kv_append", "qmm_kv_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_results_are_allocated_on_the_stream_given(lib, name):
    lib, allocated = lib
    side = binding.Stream(0x7000)
    result = _calls()[name](side)
    assert allocated and all(s is side for s in allocated)
    assert lib.calls[-1][0] == name and lib.calls[-1][1][-1] == 0x7000
    for t in result if isinstance(result, tuple) else [result]:
        assert t.read_on.cuda_stream == 0x4000
    allocated.clear()
    _calls()[name](None)
    assert allocated and all(s is None for s in allocated) and lib.calls[-1][1][-1] == 0x4000


@pytest.mark.parametrize("name,others", [("qmm_rope", ["x", "rope", "positions"]),
                                         ("qmm_kv_append", ["k", "v", "table", "lengths", "cache", "rope", "q"]),
                                         ("qmm_kv_attention", ["x", "table", "lengths", "cache"])])
def test_another_device_is_refused(lib, name, others):
    lib, _ = lib
    for other in others:
        with pytest.raises(ValueError):
            _calls(0, other)[name](None)
    with pytest.raises(ValueError, match="current device"):
        _calls(1)[name](None)
    with pytest.raises(ValueError, match="stream"):
        _calls()[name](binding.Stream(device_index=1))
    assert not lib.calls
    _calls()[name](None)
    assert len(lib.calls) == 1


def test_a_captured_call_brings_its_own_scratch(lib, monkeypatch):
    lib, allocated = lib
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(type(lib), "qmm_kv_attention_scratch", lambda self, a: 4096, raising=False)
    q._f8 = None
    _calls()["qmm_kv_attention"](None)
    args = q._ATTENTION_ARGS.unpack(lib.calls[-1][1][0])
    assert args[-1] == 4096 and args[-2] != 0


def test_shapes_and_types_are_refused(lib):
    def t(*shape, dtype=torch.bfloat16):
        return binding.on_gpu(torch.zeros(shape, dtype=dtype))
    i32 = torch.int32
    calls = _calls()
    c, r = None, None

    class Grab(Exception):
        pass
    cache = q.KvCache.__new__(q.KvCache)
    for n, v in (("heads", 2), ("page", 16), ("dim", 32), ("_at", 0x1000), ("_device", 0)):
        object.__setattr__(cache, n, v)
    rope = q.RopeTable.__new__(q.RopeTable)
    rope._at, rope._device = 0x2000, 0
    pos, tab, lens, off = t(3, dtype=i32), t(3, 4, dtype=i32), t(3, dtype=i32), t(4, dtype=i32)
    x, k = t(3, 4, 32), t(3, 2, 32)
    for bad in (lambda: q.qmm_rope(t(3, 32), rope, pos), lambda: q.qmm_rope(t(3, 4, 64)[..., ::2], rope, pos),
                lambda: q.qmm_rope(x, rope, t(4, dtype=i32)), lambda: q.qmm_rope(x, rope, t(3)), lambda: q.qmm_rope(x, rope, pos, y=t(3, 4, 16)),
                lambda: q.qmm_rope(t(3, 4, 32, dtype=torch.float64), rope, pos),
                lambda: q.qmm_kv_append(cache, t(3, 3, 32), t(3, 3, 32), tab, lens), lambda: q.qmm_kv_append(cache, k, t(2, 2, 32), tab, lens),
                lambda: q.qmm_kv_append(cache, k, k.float(), tab, lens), lambda: q.qmm_kv_append(cache, k, k, tab.long(), lens),
                lambda: q.qmm_kv_append(cache, k, k, tab[:2], lens), lambda: q.qmm_kv_append(cache, k, k, tab, lens[:2]),
                lambda: q.qmm_kv_append(cache, k, k, tab, lens, q=x), lambda: q.qmm_kv_append(cache, k, k, tab, lens, q_out=x),
                lambda: q.qmm_kv_append(cache, k, k, tab, lens, rope=rope, q=x.float()),
                lambda: q.qmm_kv_append(cache, k, k, tab, lens, rope=rope, q=x, q_out=x.float()),
                lambda: q.qmm_kv_append(cache, k, k, tab, lens, offsets=off[:3]),
                lambda: q.qmm_kv_attention(cache, t(3, 4, 16), tab, lens), lambda: q.qmm_kv_attention(cache, t(4, 4, 32), tab, lens),
                lambda: q.qmm_kv_attention(cache, x, tab, lens, y=t(3, 4, 32, dtype=torch.float64)),
                lambda: q.qmm_kv_attention(cache, x, t(4, 3, dtype=i32).t(), lens)):
        with pytest.raises(ValueError):
            bad()
    assert not lib[0].calls
    kc, sc = t(5, 2, 16, 32, dtype=torch.uint8), t(5, 2, dtype=torch.float32)
    made = q.KvCache(kc, kc, sc, sc)
    with pytest.raises(AttributeError):
        made.k = kc
    for a in ((kc.float(), kc, sc, sc), (kc, t(5, 2, 16, 16, dtype=torch.uint8), sc, sc), (kc, kc, sc[:4], sc), (kc, kc, sc, sc.double()),
              (kc[:, :, :8], kc[:, :, :8], sc, sc), (t(5, 2, 24, 32, dtype=torch.uint8),) * 2 + (sc, sc)):
        with pytest.raises(ValueError):
            q.KvCache(*a)

"""The binding of the rotation, the append and the attention: what it passes on, what it refuses before the library is
called, where its results are allocated.  On the CPU, with stand-ins."""
import math
import struct

import pytest

import binding

torch = pytest.importorskip("torch")
import mat_mul_gb300 as q  # noqa: E402

BF, I32 = torch.bfloat16, torch.int32


def t(*shape, dtype=torch.float32, index=0):
    return binding.on_gpu(torch.zeros(shape, dtype=dtype), index)


def cache(pages=6, heads=2, page=16, dim=32, index=0):
    k, v = (t(pages, heads, page, dim, dtype=torch.uint8, index=index) for _ in range(2))
    return q.KvCache(k, v, t(pages, heads, index=index), t(pages, heads, index=index))


def table(rot=32, index=0):
    return q.RopeTable(t(rot // 2, dtype=torch.int64, index=index), rot)


def rope(x=None, r=None, pos=None, **k):
    return q.qmm_rope(t(5, 4, 32, dtype=BF) if x is None else x, r or table(), t(5, dtype=I32) if pos is None else pos, **k)


def append(c=None, k=None, v=None, tab=None, lens=None, **kw):
    return q.qmm_kv_append(c or cache(), t(3, 2, 32, dtype=BF) if k is None else k, t(3, 2, 32, dtype=BF) if v is None else v,
                           t(3, 2, dtype=I32) if tab is None else tab, t(3, dtype=I32) if lens is None else lens, **kw)


def attend(c=None, x=None, tab=None, lens=None, **kw):
    return q.qmm_kv_attention(c or cache(), t(3, 4, 32, dtype=BF) if x is None else x, t(3, 2, dtype=I32) if tab is None else tab,
                              t(3, dtype=I32) if lens is None else lens, **kw)


@pytest.fixture
def lib(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    with binding.stand_in(monkeypatch) as (library, allocated):
        library.allocated = allocated
        yield library


def test_arguments(lib):
    x, pos, r = t(5, 4, 40, dtype=BF)[:, :, :32], t(5, dtype=I32), table()
    y = rope(x, r, pos, inverse=True, dtype=torch.float32)
    assert y.shape == (5, 4, 32) and y.dtype == torch.float32
    name, (args, stream) = lib.calls.pop()
    assert name == "qmm_rope" and stream == 0x4000
    assert struct.unpack("=QqQqqqqQqqqQqq", args) == (r._at, 1, pos.data_ptr(), 5, 4, 32, 2, x.data_ptr(),
                                                    160, 40, 0, y.data_ptr(), 128, 32)
    c, k, qq, off, tab = cache(), t(7, 2, 32), t(7, 4, 32), t(4, dtype=I32), t(3, 9, dtype=I32)[:, :4]
    lens = t(3, dtype=I32)
    out = append(c, k, k, tab, lens, offsets=off, rope=r, q=qq, positions=t(7, dtype=I32))
    assert out.shape == qq.shape and out.data_ptr() != qq.data_ptr()
    name, (args, _) = lib.calls.pop()
    got = struct.unpack("=QQqqQQqqqQqqQqqQQQqqqQqq", args)
    assert name == "qmm_kv_append" and got[:9] == (c._at, tab.data_ptr(), 4, 9, lens.data_ptr(), off.data_ptr(), 3, 7, 0)
    assert got[17:] == (qq.data_ptr(), 4, 128, 32, out.data_ptr(), 128, 32)
    assert append() is None and struct.unpack("=QQqqQQqqqQqqQqqQQQqqqQqq", lib.calls.pop()[1][0])[5] == 0
    y, lse = attend(c, qq, tab, lens, offsets=off, lse=True, window=8)
    name, (args, _) = lib.calls.pop()
    got = struct.unpack("=QQqqQQqqqQqqqqQqqdqqQQq", args)
    assert name == "qmm_kv_attention" and lse.shape == (7, 4) and lse.dtype == torch.float32
    assert got[9:] == (qq.data_ptr(), 4, 128, 32, 0, y.data_ptr(), 128, 32, 1.0 / math.sqrt(32), 1, 8, lse.data_ptr(), 0, 0)


@pytest.mark.parametrize("call,kw", [
    (rope, dict(x=t(5, 128))), (rope, dict(x=t(5, 4, 64)[:, :, ::2])), (rope, dict(x=t(5, 4, 32, dtype=I32))), (rope, dict(pos=t(4, dtype=I32))),
    (rope, dict(pos=t(5, dtype=torch.int64))), (rope, dict(y=t(5, 4, 16))), (rope, dict(dtype=torch.float64)), (rope, dict(pos=t(10, dtype=I32)[::2])),
    (append, dict(k=t(3, 2, 16, dtype=BF))), (append, dict(v=t(3, 3, 32, dtype=BF))), (append, dict(v=t(3, 2, 32))), (append, dict(tab=t(3, 2))),
    (append, dict(tab=t(6, dtype=I32))), (append, dict(lens=t(4, dtype=I32))), (append, dict(lens=t(3))), (append, dict(offsets=t(3, dtype=I32))),
    (append, dict(tab=t(2, 2, dtype=I32), lens=t(2, dtype=I32))), (append, dict(q=t(3, 4, 32, dtype=BF))), (append, dict(q_out=t(3, 4, 32, dtype=BF))),
    (append, dict(q=t(2, 4, 32, dtype=BF), rope=True)), (append, dict(q=t(3, 4, 32), rope=True)), (append, dict(positions=t(2, dtype=I32))),
    (append, dict(q=t(3, 4, 32, dtype=BF), rope=True, q_out=t(3, 4, 32))), (append, dict(tab=t(2, 3, dtype=I32).t())),
    (attend, dict(x=t(3, 4, 16, dtype=BF))), (attend, dict(x=t(2, 4, 32, dtype=BF))), (attend, dict(x=t(3, 4, 32, dtype=I32))),
    (attend, dict(y=t(3, 4, 16))), (attend, dict(tab=t(3, 2))), (attend, dict(lens=t(2, dtype=I32))), (attend, dict(dtype=torch.int8)),
    (attend, dict(offsets=t(4, dtype=torch.int64)))])
def test_refused(lib, call, kw):
    kw = dict(kw)
    if kw.get("rope") is True:
        kw["rope"] = table()
    with pytest.raises(ValueError):
        call(**kw)
    assert not lib.calls


@pytest.mark.parametrize("make", [
    lambda: q.KvCache(t(2, 2, 16, 32), t(2, 2, 16, 32), t(2, 2), t(2, 2)), lambda: q.KvCache(t(2, 2, 48, 32, dtype=torch.uint8), t(2, 2, 48, 32, dtype=torch.uint8), t(2, 2), t(2, 2)),
    lambda: q.KvCache(t(2, 2, 16, 40, dtype=torch.uint8), t(2, 2, 16, 40, dtype=torch.uint8), t(2, 2), t(2, 2)),
    lambda: q.KvCache(t(2, 2, 16, 32, dtype=torch.uint8), t(3, 2, 16, 32, dtype=torch.uint8), t(2, 2), t(2, 2)),
    lambda: q.KvCache(t(2, 2, 16, 32, dtype=torch.uint8), t(2, 2, 16, 32, dtype=torch.uint8), t(2, 2), t(2, 3)),
    lambda: q.RopeTable(t(16), 32), lambda: q.RopeTable(t(15, dtype=torch.int64), 32), lambda: q.qmm_rope_table(32, scaling="other"),
    lambda: q.qmm_rope_table(32, scaling="yarn"), lambda: q.qmm_rope_table(32, freqs=[1.0])])
def test_caches_and_tables_refused(lib, make):
    with pytest.raises(ValueError):
        make()
    assert not lib.calls


def test_a_cache_keeps_its_tensors(lib):
    c = cache()
    with pytest.raises(AttributeError):
        c.k = c.v


@pytest.mark.parametrize("what", ["x", "cache", "table", "lengths", "rope", "positions", "stream"])
def test_another_device_is_refused(lib, what):
    i = {what: 1}.get
    stream = binding.Stream(device_index=1) if what == "stream" else None
    calls = [lambda: rope(t(5, 4, 32, index=i("x", 0)), table(index=i("rope", 0)), t(5, dtype=I32, index=i("positions", 0)), stream=stream),
             lambda: append(cache(index=i("cache", 0)), t(3, 2, 32, index=i("x", 0)), t(3, 2, 32, index=i("x", 0)), t(3, 2, dtype=I32, index=i("table", 0)),
                            t(3, dtype=I32, index=i("lengths", 0)), rope=table(index=i("rope", 0)), positions=t(3, dtype=I32, index=i("positions", 0)),
                            stream=stream),
             lambda: attend(cache(index=i("cache", 0)), t(3, 4, 32, index=i("x", 0)), t(3, 2, dtype=I32, index=i("table", 0)),
                            t(3, dtype=I32, index=i("lengths", 0)), stream=stream)]
    takes = {"cache": calls[1:], "table": calls[1:], "lengths": calls[1:], "rope": calls[:2], "positions": calls[:2]}.get(what, calls)
    for call in takes:
        with pytest.raises(ValueError):
            call()
    assert not lib.calls


def test_results_come_from_the_calls_stream(lib):
    s = binding.Stream()
    rope(stream=s), append(q=t(3, 4, 32, dtype=BF), rope=table(), stream=s), attend(stream=s, lse=True)
    assert lib.allocated == [s] * 4 and all(args[1] == 0x5000 for _, args in lib.calls)


def test_a_captured_call_has_scratch_of_its_own(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(q, "_f8", None)
    lib.qmm_kv_attention_scratch = lambda args: 4096
    attend()
    (name, (args, _)), = lib.calls
    got = struct.unpack("=QQqqQQqqqQqqqqQqqdqqQQq", args)
    assert name == "qmm_kv_attention" and got[-1] == 4096 and got[-2] != 0

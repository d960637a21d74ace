"""The Python binding without a GPU: a library that does nothing and takes note of the calls, and tensors in host memory
that say they are on a device."""
import contextlib

import mat_mul_gb300 as q


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class Stream:
    def __init__(self, handle=0x5000, device_index=0):
        self.cuda_stream, self.device_index = handle, device_index


def on_gpu(t, index=0):
    """t as a tensor that reports to be on CUDA device `index`."""
    import torch

    class OnGpu(torch.Tensor):
        is_cuda = property(lambda self: True)

        def get_device(self):
            return index

        def record_stream(self, stream):
            self.read_on = stream
    return t.as_subclass(OnGpu)


@contextlib.contextmanager
def stand_in(monkeypatch, current_device=0):
    """The binding over a Library; yields (library, stream in use at each allocation)."""
    import torch
    lib, in_use, allocated = Library(), [None], []

    @contextlib.contextmanager
    def use(stream):
        before, in_use[0] = in_use[0], stream
        yield
        in_use[0] = before
    real = torch.empty

    def empty(*args, **kw):
        allocated.append(in_use[0])
        return on_gpu(real(*args, **kw), current_device)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(0x4000))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x4000, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current_device, raising=False)
    monkeypatch.setattr(q, "_lib", lib)
    monkeypatch.setattr(q, "_f8", None)
    yield lib, allocated


def calls(index=0):
    """(name, call(stream) on tensors of device `index`) of every call of the binding that takes a stream."""
    import torch

    def t(*shape, dtype=torch.float32):
        return on_gpu(torch.zeros(shape, dtype=dtype), index)
    u8, i32 = torch.uint8, torch.int32
    W, S = t(3, 32, 32, dtype=u8), t(3, 1, 1)
    off = t(4, dtype=i32)
    r = q.Route(t(5, 2), t(5, 2, dtype=i32), off, t(10, dtype=i32), t(5, 2, dtype=i32))
    blocks = t(4096, dtype=u8)
    return [
        ("qmm_f8_quantize", lambda s: q.qmm_f8_quantize(t(5, 32), stream=s)),
        ("qmm_f8", lambda s: q.qmm_f8(W[0], S[0], t(5, 32), stream=s)),
        ("qmm_f8_experts", lambda s: q.qmm_f8_experts(W, S, t(5, 32), off, stream=s)),
        ("qmm_route", lambda s: q.qmm_route(t(5, 3), 2, stream=s)),
        ("qmm_f8_moe", lambda s: q.qmm_f8_moe(t(5, 32), r, W, S, W, S, W, S, stream=s)),
        ("qmm", lambda s: q.qmm(q.Q8_0, blocks, 4, 32, t(5, 32), stream=s)),
        ("qmm_t", lambda s: q.qmm_t(q.Q8_0, blocks, 2, 4, 32, t(2, 5, 4), stream=s)),
        ("qmm_group", lambda s: q.qmm_group([(q.Q8_0, blocks, 4)], 32, t(5, 32), stream=s)),
        ("qmm_gate_up", lambda s: q.qmm_gate_up(q.Q8_0, blocks, q.Q8_0, blocks, 4, 32, t(5, 32), stream=s)),
        ("qmm_noalloc", lambda s: q.qmm_noalloc(q.Q8_0, blocks, 4, 32, t(5, 32), t(5, 4), stream=s)),
        ("qmm_quantize_act", lambda s: q.qmm_quantize_act(t(5, 32), stream=s)),
    ]


NAMES = ["qmm_f8_quantize", "qmm_f8", "qmm_f8_experts", "qmm_route", "qmm_f8_moe", "qmm", "qmm_t", "qmm_group",
         "qmm_gate_up", "qmm_noalloc", "qmm_quantize_act"]

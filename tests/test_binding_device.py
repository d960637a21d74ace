"""The library works on the current device: workspace, status word and launch are there.  Tensors or a stream of another
device are refused before the library is called.  On the CPU, with stand-ins."""
import pytest

import binding

pytest.importorskip("torch")


@pytest.mark.parametrize("name", binding.NAMES)
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    with binding.stand_in(monkeypatch, current_device=0) as (lib, _):
        dict(binding.calls(0))[name](None)
        assert [n for n, _ in lib.calls] == [name]
        lib.calls.clear()
        with pytest.raises(ValueError, match="current device"):
            dict(binding.calls(1))[name](None)
        assert not lib.calls
    with binding.stand_in(monkeypatch, current_device=1) as (lib, _):
        dict(binding.calls(1))[name](None)
        assert [n for n, _ in lib.calls] == [name]


@pytest.mark.parametrize("name", binding.NAMES)
def test_a_stream_of_another_device_is_refused(monkeypatch, name):
    with binding.stand_in(monkeypatch, current_device=0) as (lib, _):
        dict(binding.calls(0))[name](binding.Stream(device_index=0))
        lib.calls.clear()
        with pytest.raises(ValueError, match="stream"):
            dict(binding.calls(0))[name](binding.Stream(device_index=1))
        assert not lib.calls


def test_dequant_of_another_device_is_refused(monkeypatch):
    import mat_mul_gb300 as q
    import torch
    with binding.stand_in(monkeypatch, current_device=0) as (lib, _):
        with pytest.raises(ValueError, match="current device"):
            q.qmm_dequant(q.Q8_0, binding.on_gpu(torch.zeros(4096, dtype=torch.uint8), 1), 32)
        assert not lib.calls

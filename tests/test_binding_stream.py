"""Results that a call allocates belong to the stream that it was given, as those of any operation under
torch.cuda.stream(): memory of the current stream's pool may still be in use there when the other stream writes it, and
may be handed out again while it does.  On the CPU, with stand-ins."""
import pytest

import binding

pytest.importorskip("torch")


@pytest.mark.parametrize("name", [n for n in binding.NAMES if n != "qmm_noalloc"])   # (which allocates nothing)
def test_results_are_allocated_on_the_stream_given(monkeypatch, name):
    with binding.stand_in(monkeypatch) as (lib, allocated):
        side = binding.Stream(0x7000)
        call = dict(binding.calls())[name]
        result = call(side)
        assert allocated and all(s is side for s in allocated)
        args = lib.calls[-1][1]
        assert getattr(args[-1], "value", args[-1]) == 0x7000       # the launch is on it as well
        for t in result if isinstance(result, (tuple, list)) else [result]:
            assert t.read_on.cuda_stream == 0x4000                  # and kept until the caller's stream is done with it
        allocated.clear()
        call(None)                                                  # the current stream: nothing to switch
        assert allocated and all(s is None for s in allocated)

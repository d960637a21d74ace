"""Results on a stream that is not the current one: memory that the current stream is still writing is not given to
them."""
import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu


def test_results_on_another_stream_are_not_overwritten(cuda_lib):
    import torch
    q = cuda_lib
    rng = np.random.default_rng(2)
    W, S = (torch.from_numpy(a).cuda() for a in R.weights(rng, 400, 512))
    x = torch.from_numpy(rng.standard_normal((50, 512)).astype(np.float32)).cuda()
    logits = torch.from_numpy(rng.standard_normal((50, 16)).astype(np.float32)).cuda()
    offsets = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls = [lambda: [q.qmm_f8(W, S, x, stream=side)], lambda: list(q.qmm_f8_quantize(x, stream=side)),
             lambda: list(q.qmm_route(logits, 3, stream=side)),
             lambda: [q.qmm_f8_experts(W[None], S[None], x, offsets, stream=side)]]
    for call in calls:
        first = call()
        torch.cuda.synchronize()
        want = [t.view(torch.uint8).clone() for t in first]
        del first
        torch.cuda.synchronize()
        # blocks of the same sizes, freed with writes to them still queued behind a pause
        pause = torch.cuda.Event()
        old = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(50_000_000)
        for t in old:
            t.fill_(7)
        pause.record()
        del old, t
        got = call()
        side.synchronize()
        pause.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(want, got))


def test_results_made_on_another_stream_and_read_here(cuda_lib):
    """The same call over and over, its result read on the current stream and dropped at once."""
    import torch
    q = cuda_lib
    rng = np.random.default_rng(3)
    W, S = (torch.from_numpy(a).cuda() for a in R.weights(rng, 400, 512))
    xs = [torch.from_numpy(rng.standard_normal((50, 512)).astype(np.float32)).cuda() for _ in range(6)]
    want = [q.qmm_f8(W, S, x).double().sum() for x in xs]
    side, sums = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for x in xs:
        y = q.qmm_f8(W, S, x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(5_000_000)
        sums.append(y.double().sum())
        del y
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, sums))

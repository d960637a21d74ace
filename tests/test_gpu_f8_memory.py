"""A workspace that the GPU cannot hold: refused, and neither the caller's own operations nor the next call notice."""
import ctypes

import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu


def test_a_workspace_that_does_not_fit_is_refused_and_forgotten(cuda_lib):
    import torch
    q = cuda_lib
    rng = np.random.default_rng(0)
    W, S = (torch.from_numpy(a).cuda() for a in R.weights(rng, 200, 256))
    x = torch.from_numpy(rng.standard_normal((40, 256)).astype(np.float32)).cuda()
    want = q.qmm_f8(W, S, x)
    # the rows of the down product alone would take 2^25 * 2^16 * 4 bytes; refused before anything is launched
    some = torch.zeros(1024, device="cuda")
    p = ctypes.c_void_p(some.data_ptr())
    T, H, k = 1 << 20, 1 << 16, 32
    before = q.qmm_launch_count()
    rc = q.load().qmm_f8_moe(2, p, T, H, H, k, p, p, p, 64, 128, p, p, p, p, p, p, 2, p, H,
                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == q.QMM_ENOMEM and q.qmm_launch_count() == before
    assert torch.equal(some + 1, torch.ones_like(some))     # PyTorch asks for the runtime's last error after its launches
    torch.cuda.synchronize()
    assert torch.equal(q.qmm_f8(W, S, x), want)
    assert q.qmm_device_status() == 0

"""Offsets that fall: the groups before are whole, the ones after are skipped and reported, nothing is written twice."""
import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("scale", [1, 10])            # the product for few rows, for many
@pytest.mark.parametrize("many", [False, True])       # more experts than lanes of the warp that counts the tiles
def test_groups_that_overlap_are_skipped(cuda_lib, scale, many):
    import torch
    rng = np.random.default_rng(6)
    E, rows = (45, 30 * scale) if many else (3, 30 * scale)
    W, S = (np.stack(a) for a in zip(*(R.weights(rng, 140, 256) for _ in range(E))))
    W, S = _t(W), _t(S)
    x = _t(rng.standard_normal((rows, 256)).astype(np.float32))
    first = np.zeros(E - 3, np.int64)                 # empty groups in front
    good, bad = (np.concatenate([first, np.array(o) * scale]).astype(np.int32) for o in
                 ([0, 20, 20, 30], [0, 20, 10, 30]))
    want = cuda_lib.qmm_f8_experts(W, S, x, _t(good))
    assert cuda_lib.qmm_device_status() == 0
    y = torch.full_like(want, 7.0)
    cuda_lib.qmm_f8_experts(W, S, x, _t(bad), y=y)
    assert cuda_lib.qmm_device_status() == cuda_lib.QMM_EINDEX
    n = 20 * scale
    assert torch.equal(y[:n], want[:n]) and torch.all(y[n:] == 7.0)
    assert torch.equal(want, cuda_lib.qmm_f8_experts(W, S, x, _t(good)))
    assert cuda_lib.qmm_device_status() == 0

"""Router weights at the ends of the range: logits that are all far below zero, and infinite ones."""
import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("top", [-60.0, -87.0, -95.0, -104.0, -300.0, -700.0])
def test_sigmoid_scores_far_below_zero(cuda_lib, T, top):
    """Where every sigmoid is tiny, or below the smallest float, their quotients by the sum are not."""
    rng = np.random.default_rng(T)
    x = (top - 3 * rng.random((T, 40))).astype(np.float32)
    r = cuda_lib.qmm_route(_t(x), 5, score="sigmoid")
    w, e, *_ = R.route(x, 5, "sigmoid", True)
    assert np.array_equal(r.experts.cpu().numpy(), e)
    # two exponentials (2^-22 each), an addition and a division per score; their sum (5 terms in a tree of 5 levels);
    # a division
    got = r.weights.cpu().numpy()
    assert np.all(np.abs(got - w) <= 2 * (2 * 4 + 2 + 5 + 1) * 2.0 ** -24 * w), np.abs(got / w - 1).max()


def test_sigmoid_with_a_logit_near_zero(cuda_lib):
    """Scores of ordinary size beside tiny ones; unnormalised ones as they are."""
    x = np.array([[0.5, -3, -88.5, -100, -200, -1e30], [-80, -90, -95, -3e38, -np.inf, np.nan]], np.float32)
    for normalize in (True, False):
        r = cuda_lib.qmm_route(_t(x), 6, score="sigmoid", normalize=normalize)
        w, e, *_ = R.route(x, 6, "sigmoid", normalize)
        assert np.array_equal(r.experts.cpu().numpy(), e)
        got = r.weights.cpu().numpy()
        assert np.all(np.abs(got - w) <= 2.0 ** -19 * w + 2.0 ** -148), (got, w)


@pytest.mark.parametrize("T", [2, 300])
def test_infinite_logits(cuda_lib, T):
    """+inf is the largest logit; softmax of a row with one has no value (NaN, as its formula gives), a sigmoid of it is 1."""
    x = np.zeros((T, 9), np.float32)
    x[1, 4] = np.inf
    r = cuda_lib.qmm_route(_t(x), 3, score="sigmoid")
    assert r.experts[1].tolist() == [4, 0, 1] and np.allclose(r.weights[1].tolist(), [0.5, 0.25, 0.25], rtol=1e-6)
    for normalize in (True, False):
        r = cuda_lib.qmm_route(_t(x), 3, normalize=normalize)
        w = r.weights.cpu().numpy()
        assert r.experts[1].tolist() == [4, 0, 1] and np.isnan(w[1]).any()
        want = 1 / 3 if normalize else 1 / 9
        assert np.allclose(w[[i for i in range(T) if i != 1]], want, rtol=1e-6)

"""The gated pair's SiLU over the whole range of the gate, in both product kernels: accurate to fp32 relative to its
value, also where e^-g overflows but silu(g) * u does not vanish."""
import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu

H = I = 128
STEP = 448 * 2.0 ** -9            # gate of a code 1


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _codes(target):
    """Three codes whose values add up to about target / STEP, and the gate that they make."""
    rest, codes = np.asarray(target, np.float64) / STEP, []
    for _ in range(3):
        c = R.encode(rest)
        rest = rest - R.VALUES[c]
        codes.append(c)
    codes = np.stack(codes, 1)
    return codes, R.VALUES[codes].sum(1) * STEP


def layer(top):
    """One block of h whose gates lie within 3 below `top`: the layer's tensors, and its result with a bound."""
    codes, g = _codes(top - 3 * np.arange(I) / I)
    x = np.zeros((1, H), np.float32)
    x[0, :4] = 448                                     # scale 1, code 448
    Wg, Wu = np.zeros((I, H), np.uint8), np.zeros((I, H), np.uint8)
    Wg[:, :3] = codes
    Wu[:, 3] = 0x38                                    # u = 448 Su, which brings h near 1 or u near the top of fp32
    with np.errstate(over="ignore"):
        s = R.silu(g)
    su = 2.0 ** min(117, np.floor(-np.log2(np.abs(s).max())) - 9)
    h = s * 448 * su
    # the gate's own sum is exact but for the order of its additions; exponential 2^-22 (or half of the smallest step
    # where it is subnormal), an addition, a division and two products 2^-24 each
    e = np.abs(h) * (2.0 ** -21 + np.abs(g) * 2.0 ** -22) + np.abs(g) * 448 * su * 2.0 ** -149
    Wd = np.zeros((H, I), np.uint8)
    np.fill_diagonal(Wd, 0x38)
    one = np.ones((1, 1), np.float32)
    want, b = R.down_product(Wd, one, h[None], e[None])
    f32 = np.float32
    return x, (Wg, one * f32(2.0 ** -9), Wu, one * f32(su), Wd, one), g, want[0], b[0]


TOPS = [-97.0, -93.0, -89.0, -88.0, -87.0, -86.0, -80.0, -50.0, -20.0, -9.0, -3.0, -0.5, 3.0, 20.0, 88.0, 100.0]


@pytest.mark.parametrize("T", [3, 300])                # weights on the TMEM lanes; tokens on the lanes
@pytest.mark.parametrize("top", TOPS)
def test_silu_over_its_range(cuda_lib, T, top):
    x, weights, g, want, b = layer(top)
    assert np.all(np.abs(want) > 4 * b)                # (a result of 0 would be outside everywhere)
    route = cuda_lib.Route(_t(np.ones((T, 1), np.float32)), _t(np.zeros((T, 1), np.int32)), _t(np.array([0, T], np.int32)),
                           _t(np.arange(T, dtype=np.int32)), _t(np.arange(T, dtype=np.int32)[:, None]))
    y = cuda_lib.qmm_f8_moe(_t(np.repeat(x, T, 0)), route, *(_t(a[None]) for a in weights))
    assert cuda_lib.qmm_device_status() == 0
    y = y.cpu().numpy().astype(np.float64)
    assert np.array_equal(y, np.repeat(y[:1], T, 0))
    bad = ~(np.abs(y[0] - want) <= b)
    assert not bad.any(), (g[bad], y[0][bad], want[bad])

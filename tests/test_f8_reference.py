"""The numpy reference of the 8-bit-float operators against hand-worked values and torch's own cast."""
import numpy as np
import pytest

import f8_reference as R


def test_code_values():
    assert R.VALUES[0x00] == 0 and R.VALUES[0x01] == 2.0 ** -9 and R.VALUES[0x07] == 7 * 2.0 ** -9
    assert R.VALUES[0x08] == 2.0 ** -6 and R.VALUES[0x38] == 1.0 and R.VALUES[0x39] == 1.125
    assert R.VALUES[0x7e] == 448 and np.isnan(R.VALUES[0x7f]) and R.VALUES[0xfe] == -448


def test_encode_ties_and_ends():
    assert list(R.encode([1.0625, 1.1875, 1.0626, 500.0, -500.0, 2.0 ** -10, 3 * 2.0 ** -10, np.nan])) == \
        [0x38, 0x3a, 0x39, 0x7e, 0xfe, 0x00, 0x02, 0x7f]


def test_encode_agrees_with_torch():
    torch = pytest.importorskip("torch")
    v = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 60
    want = torch.from_numpy(v.clip(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(v), want)


def test_product_of_one_block():
    x = np.full((1, 128), 448.0, np.float32)          # scale 1, every code 448
    W = np.full((1, 128), 0x38, np.uint8)             # every weight 1 * S
    y, A = R.product(W, np.array([[0.5]], np.float32), x)
    assert y[0, 0] == 448 * 128 * 0.5 == A[0, 0]


def test_route_order_and_ties():
    w, e, off, rows, slots = R.route([[0.0, 2.0, 2.0], [-np.inf] * 3], 2, "softmax", True)
    assert e.tolist() == [[1, 2], [0, 1]] and w.tolist() == [[0.5, 0.5], [0.0, 0.0]]
    assert off.tolist() == [0, 1, 3, 4] and rows.tolist() == [1, 0, 1, 0] and slots.tolist() == [[1, 3], [0, 2]]

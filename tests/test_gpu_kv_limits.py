"""Attention over the paged cache at its limits, on every kernel that a call may go to: scales that differ from group to
group, windows near 2^31, values far apart, NaN codes in tiles that masks cut, long sequences of which no tile may be
lost."""
import math

import numpy as np
import pytest

import kv_reference as R
from test_gpu_kv import _as, _cache, _np, _t, _u8, _within

pytestmark = pytest.mark.gpu

# rows of a sequence, table width (0: as needed) and type that lead to each kernel with 2 cache heads and a group of 4
# (kv_attention.cu: up to 32 rows; 9 to 32 16-bit ones of tables of many pages; more; more fp32 ones)
KERNELS = {"few": ("bfloat16", 2, 0), "few fp32": ("float32", 3, 0), "slim": ("float16", 5, 1300), "slim bf16": ("bfloat16", 8, 1300),
           "tc": ("bfloat16", 70, 0), "tc fp16": ("float16", 70, 0), "rows": ("float32", 40, 0)}


def _i32(a):
    return _t(np.asarray(a, np.int32))


def _run(q, cache, x, batch, **k):
    y, lse = q.qmm_kv_attention(cache, x, _t(batch.table), _i32(batch.lengths), offsets=_t(batch.offsets), lse=True, **k)
    assert q.qmm_device_status() == 0
    return y, lse


@pytest.mark.parametrize("kernel", [k for k in KERNELS if not k.startswith("tc")])
def test_every_group_of_tokens_has_the_scale_of_its_page(cuda_lib, kernel):
    """Pages of 16 tokens whose scales differ by up to 2^40, in short sequences (a tile's scales are read as soon as its
    codes are there): against 64 bits, and the same bits again and again."""
    import torch
    q = cuda_lib
    dtype, new, width = KERNELS[kernel]
    rng = np.random.default_rng(70)
    lengths = [max(n, new) for n in (130, 90, 300, 17, 500, 64)]
    batch = R.Batch(rng, [new] * 6, lengths, 16, width=width)
    cache, codes, scales = _cache(q, rng, batch, 2, 64, spread=20)
    x, xv = _as(2.0 ** -18 * rng.standard_normal((batch.T, 8, 64)), dtype)
    y, lse = _run(q, cache, x, batch, dtype=torch.float32)   # (fp16 ends at 65504, these do not)
    wy, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 0.125)
    _within(_np(y), wy, R.rounded(wy, e, "float32"), "y")
    _within(_np(lse), wl, le, "lse")
    for _ in range(50):
        again = _run(q, cache, x, batch, dtype=torch.float32)
        assert torch.equal(again[0], y) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kernel", ["tc", "tc fp16"])
def test_first_tiles_come_to_where_the_shares_were_found(cuda_lib, kernel):
    """Many sequences of one tile: the first codes of a block arrive where its prefix sums were just read.  Against 64
    bits, and the same bits again and again."""
    import torch
    q = cuda_lib
    dtype, new, _ = KERNELS[kernel]
    rng = np.random.default_rng(71)
    batch = R.Batch(rng, [new] * 40, rng.integers(new, 129, 40).tolist(), 16)
    cache, codes, scales = _cache(q, rng, batch, 2, 64, spread=20)
    x, xv = _as(2.0 ** -18 * rng.standard_normal((batch.T, 8, 64)), dtype)
    y, lse = _run(q, cache, x, batch, dtype=torch.float32)   # (fp16 ends at 65504, these do not)
    wy, wl, e, le = R.attention(xv, codes[0], scales[0], codes[1], scales[1], batch, 0.125)
    _within(_np(y), wy, R.rounded(wy, e, "float32"), "y")
    _within(_np(lse), wl, le, "lse")
    for _ in range(50):
        again = _run(q, cache, x, batch, dtype=torch.float32)
        assert torch.equal(again[0], y) and torch.equal(again[1], lse)

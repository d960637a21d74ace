"""Which row groups of a grouped product are taken: none that is out of range, and no two with a row in common."""
import numpy as np
import pytest

import f8_schedule as S

BAD = [([0, 20, 10, 30], 30, [20, 0, 0], 2),         # the third group would write rows 10 .. 20 a second time
       ([0, 31, 31], 30, [0, 0], 2), ([-1, 10, 30], 30, [0, 20], 1), ([0, 20, 10], 30, [20, 0], 1),
       ([0, 1 << 30, 30], 30, [0, 0], 2), ([0, 30] * 4, 30, [30, 0, 0, 0, 0, 0, 0], 6),
       ([5, 3, 4, 6, 30], 30, [0, 0, 0, 24], 3)]


@pytest.mark.parametrize("offsets,R,rows,refused", BAD)
def test_groups_that_overlap_are_refused(offsets, R, rows, refused):
    cum, bad = S.groups(offsets, R, 1, 1)
    assert list(np.diff(cum)) == rows
    assert bad == refused


def test_groups_in_order_are_taken():
    rng = np.random.default_rng(0)
    for _ in range(200):
        E = int(rng.integers(1, 80))
        sizes = rng.integers(0, 40, E) * (rng.random(E) < 0.6)
        offsets = np.concatenate([[0], np.cumsum(sizes)]) + int(rng.integers(0, 3))
        cum, bad = S.groups(offsets, int(offsets[-1]) + int(rng.integers(0, 2)), 16, 3)
        assert bad == 0 and list(np.diff(cum)) == [3 * -(-int(n) // 16) for n in sizes]


def test_no_offsets_make_more_tiles_than_were_allowed_for():
    """Offsets that rise and fall, on the largest sizes: the number of tiles stays below R / tokens + E times nb."""
    R, tokens, nb = 1 << 22, 128, 64
    for offsets in ([0, R] * 512 + [0], [R, 0] * 512 + [R], [0, R // 2, 0, R] * 256 + [R]):
        cum, bad = S.groups(offsets, R, tokens, nb)
        assert bad > 0 and 0 <= cum[-1] <= (R // tokens + len(offsets)) * nb

"""The pieces into which the 8-bit-float products cut their work, on the CPU: every part of every tile exactly once, and
what the kernels rely on where several CTAs share a tile."""
import numpy as np
import pytest

import f8_schedule as S
import f8_shapes as shapes


def check(offsets, R, N, K, tokens, cols, G, step):
    pieces, plan = S.walk(offsets, R, N, K, tokens, cols, G, step)
    nb, kb = -(-N // cols), -(-K // 128)
    off = [0, R] if offsets is None else list(offsets)
    cta, e, nblk, row0, ntok, k0, k1, tile, cut = (pieces[:, i].astype(np.int64) for i in range(9))
    # every K block of every tile once
    tiles = plan[0]
    seen = np.zeros(tiles * kb, np.int64)
    for a, b, t in zip(k0, k1, tile):
        assert 0 <= a < b <= kb
        seen[t * kb + a:t * kb + b] += 1
    assert np.all(seen == 1)
    # every row of every group against every row block of W once
    first = {}
    for i in range(len(pieces)):
        first.setdefault(int(tile[i]), i)
        j = first[int(tile[i])]
        assert (e[i], nblk[i], row0[i], ntok[i]) == (e[j], nblk[j], row0[j], ntok[j])
    hit = np.zeros((R + 1, nb), np.int32)
    for i in first.values():
        assert 1 <= ntok[i] <= tokens and off[e[i]] <= row0[i] and row0[i] + ntok[i] <= off[e[i] + 1]
        hit[row0[i]:row0[i] + ntok[i], nblk[i]] += 1
    rows = np.zeros(R + 1, bool)
    for a, b in zip(off, off[1:]):
        rows[a:b] = True
    assert np.all(hit[rows] == 1) and not hit[~rows].any()
    # a CTA's pieces of cut tiles fit its two partial tiles: one that begins its tile, one that does not
    parts = cut >= 0
    for c in np.unique(cta[parts]):
        mine = parts & (cta == c)
        assert (k0[mine] == 0).sum() <= 1 and (k0[mine] != 0).sum() <= 1
    # the CTAs of a cut tile are exactly those that the sharers name, in K order, and only the first begins the tile
    lead = set()
    for t in np.unique(tile[parts]):
        i = np.nonzero(tile == t)[0]
        i = i[np.argsort(k0[i])]
        c0, c1 = cut[i[0]] >> 16, cut[i[0]] & 0xffff
        assert np.all(cut[i] == cut[i[0]]) and list(cta[i]) == list(range(c0, c1 + 1)) and c1 < G
        assert k0[i[0]] == 0 and np.all(k0[i[1:]] > 0)
        lead.add(int(c0))                      # the counter of the tile
    assert len(lead) == len(np.unique(tile[parts]))
    return plan


@pytest.mark.parametrize("M,N,K,launches,tokens,cols,G,step,rule", shapes.ONE_MATRIX)
def test_one_matrix(M, N, K, launches, tokens, cols, G, step, rule):
    assert S.branch(check(None, M, N, K, tokens, cols, G, step), G) == rule


@pytest.mark.parametrize("sizes,N,K,tokens,cols,G,step,rule", shapes.EXPERTS)
def test_experts(sizes, N, K, tokens, cols, G, step, rule):
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    assert S.branch(check(offsets, sum(sizes), N, K, tokens, cols, G, step), G) == rule


def layer_rules(T, k, E, H, I, sizes):
    mean = -(-T * k // E)
    wide = mean > 24
    tokens = 128 if wide else 16 if mean <= 16 else 32
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    step, G = (128 if wide else 0), shapes.SMS
    return [S.branch(check(offsets, T * k, N, K, tokens, cols, G, step), G)
            for N, K, cols in ((I, H, 128), (H, I, 256 if wide else 128))]


@pytest.mark.parametrize("T,k,E,H,I,gate_up,down", shapes.EXPERT_LAYERS)
def test_expert_layers(T, k, E, H, I, gate_up, down):
    sizes = [T * k // E + (e < T * k % E) for e in range(E)]
    assert layer_rules(T, k, E, H, I, sizes) == [gate_up, down]


def test_every_rule_is_tried_on_every_kernel():
    for cases, at in ((shapes.ONE_MATRIX, 5), (shapes.EXPERTS, 4)):
        for cols in (128, 256):
            assert {c[-1] for c in cases if c[at] == cols} == {"few", "whole", "shared"}
    for many in (False, True):
        assert {c[5] for c in shapes.EXPERT_LAYERS if (c[0] * c[1] / c[2] > 24) == many} == {"few", "whole", "shared"}


def test_shapes_at_random():
    rng = np.random.default_rng(1)
    rules = set()
    for i in range(400):
        E = int(rng.integers(1, 12)) if i % 2 else 1
        sizes = rng.integers(0, int(rng.choice([3, 40, 700])), E) * (rng.random(E) < 0.8)
        if sizes.sum() == 0:
            sizes[0] = 1
        offsets = None if E == 1 else np.concatenate([[0], np.cumsum(sizes)])
        N, K = int(np.exp(rng.uniform(4, 9.9))), 16 * int(np.exp(rng.uniform(0, 7.1)))
        G = int(rng.choice([152, 148, 76, 70, 132, 8, 1]))
        tokens, cols, step = ((16, 128, 0), (32, 128, 0), (64, 128, 0), (128, 256, 128), (256, 256, 256), (128, 128, 128))[
            int(rng.integers(6))]
        rules.add((S.branch(check(offsets, int(sizes.sum()), N, K, tokens, cols, G, step), G), cols))
    assert len(rules) == 6

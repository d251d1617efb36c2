"""Pins of the oracle for block selection, block-sparse and shared-prefix
attention (no GPU): exact rational arithmetic for the selection, the packed
attention's oracle for the attentions, and planted mistakes that must show."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import walks

SCALE = 1.0 / np.sqrt(128.0)


def _rand(S, H, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((3, S, H, 128)).astype(np.float32)
    return [(y.view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64) for y in x]  # bf16 values


@pytest.mark.parametrize("lens", [[1], [129, 40], [700]])
def test_selection_matches_rational_arithmetic(lens):
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, _ = _rand(sum(lens), 1, 3)

    def mean(x):  # exact mean, rounded once to fp32
        cols = [sum(Fraction(float(r[d])) for r in x) / len(x) for d in range(128)]
        return [Fraction(float(np.float32(float(c)))) for c in cols]
    for keep_own in (False, True):
        idx, cnt = walks.select(q, k, cu, 256, 2, keep_own)
        for i, (q0, q1, a, b) in enumerate(walks.blocks(cu, 256)):
            qm = mean(q[q0:q1, 0])
            s = [sum(x * y for x, y in zip(qm, mean(k[t:min(t + 128, b), 0]))) for t in range(a, b, 128)]
            own = {t for t in range(len(s)) if keep_own and a + 128 * t < q1 and a + 128 * t + 128 > q0}
            want = sorted(sorted(range(len(s)), key=lambda t: (t not in own, -s[t], t) if t not in own else (False, 0, t))[:2])
            assert cnt[0, i] == len(want)
            assert idx[0, i, :cnt[0, i]].tolist() == want


def test_ties_go_to_the_lower_tile_and_nan_ranks_last():
    assert walks.pick(np.array([1.0, 2.0, 2.0, 2.0]), 2) == [1, 2]
    assert walks.pick(np.array([np.nan, -np.inf, 0.0]), 2) == [1, 2]
    assert walks.pick(np.array([-0.0, 0.0, 0.0]), 1) == [0]
    assert walks.pick(np.array([5.0, 4.0, 1.0]), 2, own=range(2, 3)) == [0, 2]


def test_all_tiles_reproduce_the_packed_attention():
    lens = [300, 1, 128]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = _rand(sum(lens), 2, 4)
    o, lse = oatt.attention(q, k, v, cu, SCALE)
    nq = len(walks.blocks(cu, 256))
    idx = np.tile(np.arange(3, dtype=np.int32), (2, nq, 1))
    cnt = np.array([[3, 3, 1, 1]] * 2, dtype=np.int32)
    o2, _, lse2 = walks.sparse_attention(q, k, v, cu, 256, idx, cnt, SCALE)
    assert np.abs(o - o2).max() < 1e-12 and np.abs(lse - lse2).max() < 1e-12
    # planted: a dropped tile, and a tile counted twice, both show
    cnt[0, 0] = 2
    o3, _, lse3 = walks.sparse_attention(q, k, v, cu, 256, idx, cnt, SCALE)
    assert np.abs(lse3[0, :256] - lse[0, :256]).min() > 1e-3 and np.array_equal(lse3[1], lse2[1])


def test_empty_list_gives_zero_and_minus_infinity():
    q, k, v = _rand(130, 1, 5)
    idx, cnt = np.full((1, 1, 2), -1, dtype=np.int32), np.zeros((1, 1), dtype=np.int32)
    o, _, lse = walks.sparse_attention(q, k, v, np.array([0, 130]), 256, idx, cnt, SCALE)
    assert np.all(o == 0) and np.all(lse == -np.inf)


def test_prefix_and_document_are_one_document():
    # one document whose first 150 rows are the prefix: the other rows' output
    # is the packed attention's
    q, k, v = _rand(200, 2, 6)
    o, lse = oatt.attention(q, k, v, np.array([0, 200]), SCALE)
    o2, wv, lse2 = walks.prefix_attention(q[150:], k[150:], v[150:], k[:150], v[:150], np.array([0, 50]), SCALE)
    assert np.abs(o[150:] - o2).max() < 1e-12 and np.abs(lse[:, 150:] - lse2).max() < 1e-12
    assert np.all(wv >= np.abs(o2) - 1e-12)


def test_prefix_documents_do_not_see_each_other():
    q, k, v = _rand(60, 1, 7)
    cu = np.array([0, 20, 60])
    before = walks.prefix_attention(q[10:], k[10:], v[10:], k[:10], v[:10], cu - [0, 0, 10], SCALE)[0]
    k[40:], v[40:] = 3.0, -3.0  # rows of the second document
    after = walks.prefix_attention(q[10:], k[10:], v[10:], k[:10], v[:10], cu - [0, 0, 10], SCALE)[0]
    assert np.array_equal(before[:20], after[:20]) and not np.array_equal(before[20:], after[20:])

"""Work lists of the block-sparse and shared-prefix forwards, built on the host
through h3attn_walk_list_host (no GPU), and the calls' refusals that need none.

Checked for every layout: each (row, head) is finished exactly once, by one
segment or by one join record; the key tiles that reach it are its whole walk,
each once; partial rows are used once and inside the count; no segment holds
rows of a document that its own tiles do not belong to; the pairs are evenly
loaded."""
import math

import numpy as np
import pytest

from packed_varlen_non_gb300 import h3attn as H

VARLEN = [1400, 2576, 2400, 488, 3416, 1512, 3168, 1600, 1928, 1248, 3440, 800, 2088, 1760, 2328, 2616]
LAYOUTS = [
    ([1], 1), ([1] * 40, 3), ([20423], 21), ([64, 80], 2), (VARLEN, 21), ([31, 32, 33, 1, 511, 512, 513, 2], 2),
    ([600] * 30, 5), ([700, 5, 5000, 3, 3, 129], 4), ([4096, 4096, 4096], 21), ([16320, 5033], 56),
]


def tiles(n):
    return math.ceil(n / 128)


def check_rows(lens, heads, units, off, joins, part_rows, walk_of, share_of):
    """walk_of(row) -> number of steps of the row's walk; share_of(segment) ->
    its steps of that walk as a (lo, hi) range."""
    S = sum(lens)
    assert off[0] == 0 and off[-1] == len(units) and np.all(np.diff(off) >= 1)
    done = np.zeros((heads, S), dtype=np.int32)
    by_part = {}
    used = np.zeros(part_rows, dtype=np.int32)
    for s in units:
        q0, q1, _, _, h, _, _, part = (int(x) for x in s)
        assert 0 <= q0 < q1 <= S and q1 - q0 <= 512 and 0 <= h < heads
        if part < 0:
            done[h, q0:q1] += 1
            assert share_of(s) == (0, walk_of(q0)) and walk_of(q0) == walk_of(q1 - 1)
        else:
            used[part:part + q1 - q0] += 1
            by_part[part] = s
    assert np.all(used == 1)
    for r0, r1, h, key_lo, a_part, a_rows, n_a, a_q0, b_part, b_rows, n_b, b_q0, key_hi, *_ in joins.tolist():
        assert 0 <= r0 < r1 <= S
        done[h, r0:r1] += 1
        spans = []
        for part, rows, n, q0 in ((a_part, a_rows, n_a, a_q0), (b_part, b_rows, n_b, b_q0)):
            for c in range(n):
                s = by_part[part + c * rows]
                assert int(s[0]) == q0 and int(s[1]) - q0 == rows and int(s[4]) == h
                assert q0 <= r0 and r1 <= q0 + rows
                spans.append(share_of(s))
        if key_hi > key_lo:  # the join attends to the document itself
            cu = np.concatenate([[0], np.cumsum(lens)])
            d = int(np.searchsorted(cu, r0, side="right")) - 1
            assert (key_lo, key_hi) == (cu[d], cu[d + 1]) and key_hi - key_lo <= 32
            spans.append((walk_of(r0) - tiles(key_hi - key_lo), walk_of(r0)))
        spans.sort()
        assert spans[0][0] == 0 and spans[-1][1] == walk_of(r0) == walk_of(r1 - 1)
        assert all(x[1] == y[0] for x, y in zip(spans, spans[1:]))
    assert np.all(done == 1)


@pytest.mark.parametrize("lens,heads", LAYOUTS)
@pytest.mark.parametrize("q_block,max_blocks", [(256, 20), (512, 40), (512, 1)])
@pytest.mark.parametrize("pairs", [76, 5])
def test_list_walk_covers_every_row(lib, lens, heads, q_block, max_blocks, pairs):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    units, off, joins, part_rows = H.h3attn_walk_list_host(0, cu, heads, q_block, max_blocks, pairs)
    blocks = [(r, min(r + q_block, b), a, b) for a, b in zip(cu[:-1], cu[1:]) for r in range(a, b, q_block)]
    for s in units:
        q0, q1, b, e, _, block, _, _ = (int(x) for x in s)
        assert blocks[block] == (q0, q1, b, e)
    # a piece's share of a list of n entries is [n i / m, n (i + 1) / m): any n is partitioned
    n = 20160

    def share(s):
        i, m = int(s[6]) & 0xffff, (int(s[6]) >> 16) & 0xffff
        assert 0 <= i < m
        return n * i // m, n * (i + 1) // m
    check_rows(lens, heads, units, off, joins, part_rows, lambda row: n, share)


@pytest.mark.parametrize("lens,heads", LAYOUTS)
@pytest.mark.parametrize("prefix", [1, 128, 2430, 12960])
@pytest.mark.parametrize("pairs", [76, 5])
def test_prefix_walk_covers_every_row(lib, lens, heads, prefix, pairs):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    units, off, joins, part_rows = H.h3attn_walk_list_host(1, cu, heads, prefix, 0, pairs)
    tp = tiles(prefix)
    doc = np.repeat(np.arange(len(lens)), lens)
    steps = tp + np.array([tiles(n) for n in lens])[doc]
    for s in units:
        q0, q1, b, e, _, lo, hi, _ = (int(x) for x in s)
        assert 0 <= lo < hi
        if hi > tp:  # own tiles: rows of one document, whose bounds the segment has
            assert doc[q0] == doc[q1 - 1] and (b, e) == (cu[doc[q0]], cu[doc[q0] + 1])
    check_rows(lens, heads, units, off, joins, part_rows, lambda row: int(steps[row]), lambda s: (int(s[5]), int(s[6])))


def cost(s, lo, hi):
    return hi - lo + 1 + (int(s[7]) >= 0)


@pytest.mark.parametrize("lens,heads,prefix", [([4096] * 3, 21, 2430), ([1] * 32, 21, 5033), ([20423], 21, 405)])
def test_prefix_passes_are_shared_and_pairs_evenly_loaded(lib, lens, heads, prefix):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    units, off, _, _ = H.h3attn_walk_list_host(1, cu, heads, prefix, 0, 76)
    tp = tiles(prefix)
    # steps over the prefix: no more than one pass per 512 rows of a head, rounded up per document of 512 or more
    steps = sum(min(int(s[6]), tp) - min(int(s[5]), tp) for s in units)
    passes = math.ceil(sum(lens) / 512) if max(lens) < 512 else sum(math.ceil(n / 512) for n in lens)
    assert steps <= heads * passes * tp
    loads = [sum(cost(s, int(s[5]), int(s[6])) for s in units[off[p]:off[p + 1]]) for p in range(len(off) - 1)]
    assert max(loads) <= 1.15 * sum(loads) / 76 + 2


def _status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


def test_host_listing_rejects_bad_arguments(lib):
    ok = (0, [0, 10], 2, 256, 1, 4)
    H.h3attn_walk_list_host(*ok)
    for bad in [(2, [0, 10], 2, 256, 1, 4), (0, [0, 10], 2, 128, 1, 4), (0, [0, 10], 2, 256, 0, 4),
                (0, [0, 10], 2, 256, (1 << 20) + 1, 4), (1, [0, 10], 2, 0, 0, 4), (1, [0, 10], 2, -5, 0, 4),
                (0, [0, 10, 10], 2, 256, 1, 4), (0, [0, 10], 0, 256, 1, 4), (0, [0, 10], 2, 256, 1, 0),
                (1, [1, 10], 2, 5, 0, 4), (1, [0], 2, 5, 0, 4)]:
        assert _status(lambda: H.h3attn_walk_list_host(*bad)) == H.H3ATTN_EINVAL, bad


def test_calls_reject_a_null_plan(lib):
    E = H.H3ATTN_EINVAL
    assert _status(lambda: H.h3attn_plan_set_sparse(None, 256, 4, stream=0)) == E
    assert _status(lambda: H.h3attn_plan_sparse_info(None)) == E
    assert _status(lambda: H.h3attn_plan_set_prefix(None, 4, stream=0)) == E
    assert _status(lambda: H.h3attn_block_select(None, 16, 16, 1, 16, 16, qkv_row_stride=128, stream=0)) == E
    assert _status(lambda: H.h3attn_forward_sparse(None, 16, 16, 16, 16, 16, 16, 0.1, qkv_row_stride=128,
                                                   o_row_stride=128, stream=0)) == E
    assert _status(lambda: H.h3attn_forward_prefix(None, 16, 16, 16, 16, 16, 16, 0.1, qkv_row_stride=128,
                                                   prefix_row_stride=128, o_row_stride=128, stream=0)) == E

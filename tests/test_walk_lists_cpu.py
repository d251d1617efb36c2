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
    ([1], 1), ([1] * 40, 3), ([1] * 200, 2), ([32, 1, 7, 30] * 6, 3), ([1] * 300, 21), ([32, 30, 2], 7), ([20423], 21), ([64, 80], 2), (VARLEN, 21), ([31, 32, 33, 1, 511, 512, 513, 2], 2),
    ([600] * 30, 5), ([1, 2672, 2210, 4, 2379], 2), ([700, 5, 5000, 3, 3, 129], 4), ([4096, 4096, 4096], 21), ([16320, 5033], 56),
]


def tiles(n):
    return math.ceil(n / 128)


def check_rows(lens, heads, units, off, joins, part_rows, steps_of, share_of):
    """steps_of(segment) -> steps of its whole walk; share_of(segment) -> those it
    takes, as a (lo, hi) range.  Returns (row, head) -> keys the join attends to."""
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
            assert share_of(s) == (0, steps_of(s))
        else:
            used[part:part + q1 - q0] += 1
            by_part[part] = s
    assert np.all(used == 1)
    inline = {}
    for r0, r1, h, q0, part, rows, n, key_lo, key_hi, *rest in joins.tolist():
        assert 0 <= r0 < r1 <= S and r1 - r0 <= 8 and n >= 1 and rest == [0, 0, 0]
        done[h, r0:r1] += 1
        spans = []
        for c in range(n):
            s = by_part[part + c * rows]
            assert int(s[0]) == q0 and int(s[1]) - q0 == rows and int(s[4]) == h
            assert q0 <= r0 and r1 <= q0 + rows
            spans.append(share_of(s))
        assert spans[0][0] == 0 and spans[-1][1] == steps_of(s)
        assert all(x[1] == y[0] for x, y in zip(spans, spans[1:]))
        if key_hi > key_lo:
            for r in range(r0, r1):
                inline[h, r] = (key_lo, key_hi)
    assert np.all(done == 1)
    return inline


@pytest.mark.parametrize("lens,heads", LAYOUTS)
@pytest.mark.parametrize("q_block,max_blocks", [(256, 20), (512, 40), (512, 1)])
@pytest.mark.parametrize("pairs", [76, 5])
def test_list_walk_covers_every_row(lib, lens, heads, q_block, max_blocks, pairs):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    units, off, joins, own, part_rows = H.h3attn_walk_list_host(0, cu, heads, q_block, max_blocks, pairs)
    blocks = [(r, min(r + q_block, b), a, b) for a, b in zip(cu[:-1], cu[1:]) for r in range(a, b, q_block)]
    for s in units:
        q0, q1, b, e, _, block, _, _ = (int(x) for x in s)
        assert blocks[block][0] <= q0 < q1 <= blocks[block][1] and blocks[block][2:] == (b, e)
    # a piece's share of a list of n entries is [n i / m, n (i + 1) / m): any n is partitioned
    n = 20160

    def share(s):
        i, m = int(s[6]) & 0xffff, (int(s[6]) >> 16) & 0xffff
        assert 0 <= i < m
        return n * i // m, n * (i + 1) // m
    assert not check_rows(lens, heads, units, off, joins, part_rows, lambda s: n, share) and len(own) == 0


@pytest.mark.parametrize("lens,heads", LAYOUTS)
@pytest.mark.parametrize("prefix", [1, 128, 2430, 12960])
@pytest.mark.parametrize("pairs", [76, 5])
def test_prefix_walk_covers_every_row(lib, lens, heads, prefix, pairs):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    units, off, joins, own, part_rows = H.h3attn_walk_list_host(1, cu, heads, prefix, 0, pairs)
    tp = tiles(prefix)
    doc = np.repeat(np.arange(len(lens)), lens)

    def steps(s):
        return tp + (tiles(int(s[3]) - int(s[2])) if s[3] > 0 else -int(s[3]))
    inline = check_rows(lens, heads, units, off, joins, part_rows, steps, lambda s: (int(s[5]), int(s[6])))
    for h, r in inline:
        assert inline[h, r] == (cu[doc[r]], cu[doc[r] + 1]) and lens[doc[r]] <= 32
    seen = set()
    for s in units:
        q0, q1, b, e, h, lo, hi, part = (int(x) for x in s)
        assert 0 <= lo < hi <= steps(s)
        if e > 0:  # rows of one document, whose bounds the segment has
            assert doc[q0] == doc[q1 - 1] and (b, e) == (cu[doc[q0]], cu[doc[q0] + 1])
            continue
        assert lo < tp  # every piece begins in the prefix
        if (h, q0) in seen:
            continue
        seen.add((h, q0))
        # the own tiles are exactly those of each row's document, unless the join has it
        want, at = [], q0
        while at < q1:
            d = doc[at]
            end = min(int(cu[d + 1]), q1)
            if (h, at) not in inline:
                want += [(t, int(cu[d + 1]) - t, at - q0, end - q0) for t in range(cu[d], cu[d + 1], 128)]
            at = end
        table = own[b:b - e]
        assert [tuple(x) for x in table[:, :4].tolist()] == want
        for t in table:  # lanes of the other documents' rows, 32 a word
            rows = np.arange(512)
            skip = (rows < t[2]) | (rows >= t[3])
            words = t[4:].astype(np.uint32)
            assert np.array_equal((words[rows // 32] >> (rows % 32).astype(np.uint32)) & 1, skip)


def cost(s, lo, hi):
    return hi - lo + 3 + (int(s[7]) >= 0)  # about: two streams' segments have less of a fixed cost


@pytest.mark.parametrize("lens,heads,prefix", [([4096] * 3, 21, 2430), ([1] * 32, 21, 5033), ([20423], 21, 405)])
def test_prefix_passes_are_shared_and_pairs_evenly_loaded(lib, lens, heads, prefix):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    units, off, _, _, _ = H.h3attn_walk_list_host(1, cu, heads, prefix, 0, 76)
    tp = tiles(prefix)
    # steps over the prefix: one pass per 512 rows of a head, or per 256 where two streams run side by side
    steps = sum(min(int(s[6]), tp) - min(int(s[5]), tp) for s in units)
    rows = 512 if max(int(s[1]) - int(s[0]) for s in units) > 256 else 256
    assert steps in (heads * math.ceil(sum(lens) / rows) * tp, heads * sum(math.ceil(n / rows) for n in lens) * tp)
    loads = [sum(cost(s, int(s[5]), int(s[6])) for s in units[off[p]:off[p + 1]]) for p in range(len(off) - 1)]
    assert max(loads) <= 1.15 * sum(loads) / 76 + 4


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

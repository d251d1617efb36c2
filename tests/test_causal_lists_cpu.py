"""Work lists of the causal forward, built on the host (no GPU), and the calls'
refusals that need none.

Checked for every layout: each (token, head) is finished exactly once, by one
segment or by one join record; the key tiles that reach it begin with its
document and end behind the token itself; partial rows are used once and inside
the count; the pairs are evenly loaded."""
import math

import numpy as np
import pytest

from packed_varlen_non_gb300 import h3attn as H

VARLEN = [1400, 2576, 2400, 488, 3416, 1512, 3168, 1600, 1928, 1248, 3440, 800, 2088, 1760, 2328, 2616]
LAYOUTS = [([1], 1, 1), ([1] * 40, 4, 2), ([64, 80], 8, 2), ([20423], 28, 4), (VARLEN, 21, 21), (VARLEN, 32, 4), ([700, 5, 129], 10, 2),
           ([511, 512, 513, 1], 6, 1), ([5000], 1, 1), ([12000], 34, 2), ([300] * 9, 17, 1), ([4096], 64, 2), ([2049], 48, 2)]


def pack_of(group):
    return max(p for p in range(1, 17) if group % p == 0)


@pytest.mark.parametrize("lens,heads,kv", LAYOUTS)
@pytest.mark.parametrize("pairs", [76, 5])
def test_every_token_and_head_is_covered(lib, lens, heads, kv, pairs):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    doc = np.repeat(np.arange(len(lens)), lens)
    pack = pack_of(heads // kv)
    units, off, joins, own, part_rows = H.h3attn_walk_list_host(2, cu, heads, kv, 0, pairs)
    assert off[0] == 0 and off[-1] == len(units) and np.all(np.diff(off) >= 1) and len(own) == 0
    done = np.zeros((heads, cu[-1]), dtype=np.int32)
    used, by_part = np.zeros(part_rows, dtype=np.int32), {}
    for u in units:
        q0, q1, b, e, h, lo, hi, part = (int(x) for x in u)
        assert 0 <= q0 < q1 and q1 - q0 <= 4 * (128 // pack) and 0 <= h and h + pack <= heads and h % pack == 0
        assert h // (heads // kv) == (h + pack - 1) // (heads // kv)  # one key head
        assert (b, e) == (cu[doc[q0]], cu[doc[q0] + 1]) and q1 <= e
        last = math.ceil((q1 - b) / 128)
        assert 0 <= lo < hi <= last
        if part < 0:
            assert (lo, hi) == (0, last)
            done[h:h + pack, q0:q1] += 1
        else:
            used[part:part + pack * (q1 - q0)] += 1
            by_part[part] = u
    assert np.all(used == 1)
    for r0, r1, h, q0, part, rows, n, key_lo, key_hi, *rest in joins.tolist():
        assert r0 < r1 <= r0 + 8 and n >= 2 and key_lo == key_hi == 0 and rest == [0, 0, 0]
        done[h, r0:r1] += 1
        at = 0
        for c in range(n):
            # piece c's rows of head h begin at the segment's own first partial row and (h - head) tokens further
            base = max(p for p in by_part if p <= part + c * rows)
            u = by_part[base]
            assert int(u[0]) == q0 and rows == pack * (int(u[1]) - q0) and r1 <= int(u[1])
            assert part + c * rows - base == (h - int(u[4])) * (int(u[1]) - q0) and 0 <= h - int(u[4]) < pack
            assert int(u[5]) == at
            at = int(u[6])
        assert at == math.ceil((int(u[1]) - int(u[2])) / 128)
    assert np.all(done == 1)


def test_the_pairs_are_evenly_loaded(lib):
    # (long enough that a segment's and a piece's fixed costs do not decide)
    for lens, heads, kv in (([20423], 28, 4), (VARLEN, 32, 4), (VARLEN, 21, 21)):
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        units, off, _, _, _ = H.h3attn_walk_list_host(2, cu, heads, kv, 0, 76)
        load = [int(sum(units[a:b, 6] - units[a:b, 5])) for a, b in zip(off[:-1], off[1:])]
        assert len(load) == 76 and max(load) <= 1.15 * np.mean(load) + 4


def status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


def test_refusals(lib):
    E = H.H3ATTN_EINVAL
    for kv in (0, -1, 3, 8):
        assert status(lambda: H.h3attn_walk_list_host(2, [0, 10], 4, kv, 0, 76)) == E
    assert status(lambda: H.h3attn_walk_list_host(2, [0, 2 ** 31 - 1], 1, 1, 0, 76)) == E
    assert status(lambda: H.h3attn_plan_set_causal(None, 1, stream=0)) == E
    assert status(lambda: H.h3attn_forward_causal(None, 16, 16, 16, 16, 0.1, q_row_stride=128, kv_row_stride=128, o_row_stride=128,
                                                  stream=0)) == E

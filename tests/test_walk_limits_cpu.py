"""The host listing of the sparse and prefix forwards' work at the end of its
32-bit row numbers (no GPU, no tensors: only the layout is that long)."""
import numpy as np
import pytest

from packed_varlen_non_gb300 import h3attn as H

MOST = 2 ** 31 - 1 - 512


@pytest.mark.parametrize("kind,p0,p1", [(0, 256, 4), (0, 512, 4), (1, 100, 0)])
@pytest.mark.parametrize("cu", [[0, 2 ** 31 - 1], [0, MOST + 1], [0, 2 ** 31 - 200, 2 ** 31 - 1], [0, 100, MOST + 1]])
def test_longer_layouts_are_refused(lib, kind, p0, p1, cu):
    with pytest.raises(H.H3AttnError) as e:
        H.h3attn_walk_list_host(kind, cu, 1, p0, p1, 76)
    assert e.value.status == H.H3ATTN_EINVAL and "too many tokens" in str(e.value)


def test_the_longest_layout_is_covered(lib):
    units, off, joins, own, _ = H.h3attn_walk_list_host(0, [0, MOST], 1, 512, 1, 76)
    rows = units[np.argsort(units[:, 0], kind="stable")].astype(np.int64)
    assert rows[0, 0] == 0 and rows[-1, 1] == MOST and np.all(rows[1:, 0] == rows[:-1, 1])
    assert np.all((rows[:, 1] - rows[:, 0] <= 512) & (rows[:, 5] == rows[:, 0] // 512) & (rows[:, 7] == -1))

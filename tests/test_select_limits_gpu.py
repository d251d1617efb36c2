"""Block selection at the sizes where its launch changes, each the first
selection of a process of its own (what an earlier, larger call has set must
not matter), against the fp64 oracle."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import sys
import numpy as np
from oracle import walks
from tests import walk_cases as W

tiles = int(sys.argv[1])
n = 128 * tiles - 5
s = W.Sparse([n], 1, 512, 16)
q, k = W.rows(n, 1, 1), W.rows(n, 1, 2)
idx, cnt = s.select(q, k, 16, keep_own=True)
# the oracle's rule, the tiles' means computed once
means = [[x[i:i + b].mean(axis=0).astype(np.float32).astype(np.float64) for i in range(0, n, b)]
         for x, b in ((W.f64(q)[:, 0], 512), (W.f64(k)[:, 0], 128))]
score = np.array(means[0]) @ np.array(means[1]).T
assert idx.shape == (1, len(score), 16) and np.all(cnt == 16)
for i, line in enumerate(score):
    own = range(4 * i, min(4 * i + 4, tiles))
    assert idx[0, i].tolist() == walks.pick(line, 16, own), i
"""


# 352 tiles: 49,152 bytes of dynamic shared memory and a few static ones; more
# than 1,536 tiles: fewer than eight query blocks a thread block
@pytest.mark.parametrize("tiles", [351, 352, 353, 1536, 1537, 2100])
def test_first_selection_of_a_process(lib, tiles):
    r = subprocess.run([sys.executable, "-c", CHILD, str(tiles)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]

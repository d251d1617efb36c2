"""What a plan's device error word says when both of its events have happened
before it is read: a bounded wait that ran out (outputs invalid) outweighs a
listed key tile outside its document (the tile skipped)."""
import numpy as np
import pytest

from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W

WAIT_NS = 1_000_000


def status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


@pytest.mark.gpu
@pytest.mark.parametrize("q_block,lens", [(256, [300, 500]), (512, [38912])])  # two streams a pair, and one
@pytest.mark.parametrize("order", ["wait", "tile", "wait tile", "tile wait", "tile wait tile"])
def test_a_timeout_outweighs_a_skipped_tile(lib, q_block, lens, order):
    s = W.Sparse(lens, 1, q_block, 40)
    q, k, v = (W.rows(s.S, 1, 1 + i) for i in range(3))
    idx = np.zeros((1, s.nq, 40), dtype=np.int32)
    idx[:, :, -1] = 1 << 20
    s.lists(idx, np.full((1, s.nq), 40, dtype=np.int32))
    for event in order.split():
        if event == "wait":
            H.h3attn_selftest_plan_wait(s.plan.handle, WAIT_NS)
        else:
            s.forward(q, k, v)
    assert status(lambda: W.ok(s.plan)) == (H.H3ATTN_ETIMEOUT if "wait" in order else H.H3ATTN_EINVAL)
    W.ok(s.plan)  # read once


def test_refusals(lib):
    assert status(lambda: H.h3attn_selftest_plan_wait(None, WAIT_NS, stream=0)) == H.H3ATTN_EINVAL

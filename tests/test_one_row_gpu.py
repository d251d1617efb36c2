"""A single token: one row has no stride, so whatever its tensors' row strides say,
the calls answer as they do for rows one behind the other."""
import pytest
import torch

from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.test_causal_gpu import Causal
from tests.test_tree_gpu import Tree

pytestmark = pytest.mark.gpu

STRIDES = [1 << 38, 1 << 39, (1 << 45) + 8, (1 << 62) - 8]


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("heads,kv", [(8, 2), (7, 1)])
def test_one_token_over_a_cache(lib, heads, kv, stride):
    t = Tree([300], [1], heads, kv, 16)
    o, lse = t.forward()
    o2, lse2 = W.outputs(1, heads)
    H.h3attn_forward_tree(t.plan.handle, t.q.data_ptr(), t.cache, t.d_table, t.d_ctx, o2.data_ptr(), W.SCALE, lse2, q_row_stride=stride,
                          o_row_stride=stride)
    W.ok(t.plan)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("heads,kv", [(8, 2), (7, 1)])
def test_a_prompt_of_one_token(lib, heads, kv, stride):
    c = Causal([1], heads, kv)
    q, k, v = c.inputs(1)
    o, lse = c.forward(q, k, v)
    o2, lse2 = W.outputs(1, heads)
    H.h3attn_forward_causal(c.plan.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), W.SCALE, lse2, q_row_stride=stride,
                            kv_row_stride=stride, o_row_stride=stride)
    W.ok(c.plan)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)

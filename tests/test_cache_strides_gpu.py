"""The tree forward over caches whose strides come in any order and with room between
rows, heads and pages."""
import pytest
import torch

from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.test_tree_gpu import Tree, random_masks

pytestmark = pytest.mark.gpu


def laid_out(x, order, room):
    """A copy of x [pages, tokens, heads, 128] whose dimensions lie in the given order, the first outermost, each with `room` elements behind it."""
    strides, step = [0, 0, 0, 1], 128 + room
    for d in reversed(order):
        strides[d] = step
        step = step * x.shape[d] + room
    buf = torch.full((step,), float("nan"), dtype=x.dtype, device="cuda")
    y = buf.as_strided(x.shape, strides)
    y.copy_(x)
    return y


@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)])
@pytest.mark.parametrize("room", [0, 8, 136])
@pytest.mark.parametrize("ctx,drafts,heads,kv,page", [([300, 5, 77], [4, 1, 16], 6, 2, 16), ([130] * 100, [1] * 100, 8, 2, 24), ([500], [64], 5, 1, 136)])
def test_strides_in_any_order(lib, ctx, drafts, heads, kv, page, order, room):
    t = Tree(ctx, drafts, heads, kv, page)
    masks = random_masks(drafts, 3)
    o, lse = t.forward(masks)
    W.ok(t.plan)
    t.check(o, lse, masks)
    cache = H.Cache(laid_out(t.kc, order, room), laid_out(t.vc, order, room))
    o2, lse2 = t.forward(masks, cache=cache)
    W.ok(t.plan)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)

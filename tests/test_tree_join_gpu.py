"""The join of the tree forward by itself: on a workspace that no forward has
written it writes nothing, whatever the memory held before; entries that name
slots the workspace has not are left out; and behind a forward it gives the same
bits again."""
import pytest
import torch

from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d
from tests.test_tree_gpu import Tree

# drafts, heads, key heads, sequences: a row a block, a row a warp, two rows a warp, two ranges a block, two query tiles
SHAPES = [(1, 8, 2, 1), (4, 28, 4, 16), (16, 28, 4, 40), (1, 32, 8, 40), (64, 64, 8, 2)]


def status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


def items_of(drafts, heads, kv, docs):
    group = heads // kv
    pack = max(p for p in range(1, 129) if group % p == 0)
    toks = min(128 // pack, drafts)
    return docs * kv * ((group // pack * -(-drafts // toks) + 1) // 2)


@pytest.mark.gpu
@pytest.mark.parametrize("drafts,heads,kv,docs", SHAPES)
def test_a_fresh_workspace_has_nothing_to_join(lib, drafts, heads, kv, docs):
    # memory full of large numbers goes back to the device first, in blocks of the sizes that the plan asks for
    dirty = [torch.full((n,), 0x3F7F7F7F, dtype=torch.int32, device="cuda") for n in [1 << 12] * 512 + [1 << 18] * 128 + [1 << 24] * 4]
    del dirty
    torch.cuda.empty_cache()
    with H.Plan(docs_1d([drafts] * docs), heads) as plan:
        H.h3attn_plan_set_tree(plan.handle, kv)
        o, lse = W.outputs(drafts * docs, heads)
        o.fill_(5.0), lse.fill_(7.0)
        H.h3attn_selftest_tree_join(plan.handle, o, lse)
        torch.cuda.synchronize()
        assert torch.all(o == 5.0) and torch.all(lse == 7.0)
        W.ok(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("drafts,heads,kv,docs", SHAPES)
def test_entries_outside_the_workspace_are_left_out(lib, drafts, heads, kv, docs):
    with H.Plan(docs_1d([drafts] * docs), heads) as plan:
        H.h3attn_plan_set_tree(plan.handle, kv)
        n, sms = items_of(drafts, heads, kv, docs), torch.cuda.get_device_properties(0).multi_processor_count
        slots = 2 * sms * (2 if n > sms and drafts * heads // kv <= 128 else 1)
        top = 2 ** 31 - 1
        bad = [(slots, 2), (slots - 1, 2), (slots - 2, 2), (-1, 2), (-2 ** 31, 2), (top, 2), (top - 1, top), (0, top), (1, slots),
               (0, slots // 2 + 1), (2, slots // 2), (0, -5), (0, -2 ** 31), (0, 0), (3, 1), (top, 1)]
        o, lse = W.outputs(drafts * docs, heads)
        o.fill_(5.0), lse.fill_(7.0)
        for i in range(0, len(bad), n):
            line = [bad[(i + j) % len(bad)] for j in range(n)]
            H.h3attn_selftest_tree_join(plan.handle, o, lse, joins=torch.tensor(line, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert torch.all(o == 5.0) and torch.all(lse == 7.0)
        # the last slots that there are
        good = torch.tensor([[0, slots // 2]] * n, dtype=torch.int32, device="cuda")
        H.h3attn_selftest_tree_join(plan.handle, o, lse, joins=good)
        torch.cuda.synchronize()
        W.ok(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("drafts,heads,kv,docs", SHAPES)
def test_the_join_repeats_itself(lib, drafts, heads, kv, docs):
    t = Tree([2000 + 37 * i for i in range(docs)], [drafts] * docs, heads, kv, 64)
    o, lse = t.forward()
    t.check(o, lse)
    o2, lse2 = torch.full_like(o, 5.0), torch.full_like(lse, 7.0)
    H.h3attn_selftest_tree_join(t.plan.handle, o2, lse2)
    joined = lse2 != 7.0
    assert joined.any()
    assert torch.equal(o2[joined.T], o[joined.T]) and torch.equal(lse2[joined], lse[joined])
    assert torch.all(o2[~joined.T] == 5.0)
    W.ok(t.plan)


@pytest.mark.gpu
def test_refusals(lib):
    E = H.H3ATTN_EINVAL
    with H.Plan(docs_1d([3, 4]), 4) as plan:
        o, lse = W.outputs(7, 4)
        assert status(lambda: H.h3attn_selftest_tree_join(plan.handle, o, o_row_stride=512)) == E  # no workspace
        H.h3attn_plan_set_tree(plan.handle, 2)
        H.h3attn_selftest_tree_join(plan.handle, o, lse)
        four = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
        H.h3attn_selftest_tree_join(plan.handle, o, lse, joins=four)
        for kw in (dict(joins=four[:3]), dict(o=o.data_ptr() + 8, o_row_stride=512), dict(o=None, o_row_stride=512),
                   dict(o=o.data_ptr(), o_row_stride=504), dict(lse=lse.data_ptr() + 2)):
            assert status(lambda: H.h3attn_selftest_tree_join(plan.handle, **{**dict(o=o, lse=lse), **kw})) == E, kw
        for bad in (four.long(), four.cpu(), four.T, four[0]):
            with pytest.raises(ValueError):
                H.h3attn_selftest_tree_join(plan.handle, o, lse, joins=bad)
        torch.cuda.synchronize()


def test_a_null_plan_is_refused(lib):
    assert status(lambda: H.h3attn_selftest_tree_join(None, 16, o_row_stride=128, stream=0)) == H.H3ATTN_EINVAL

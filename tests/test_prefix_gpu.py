"""The shared-prefix forward on the GPU, against the fp64 oracle: batches from
one single-token document on, prefixes from one row on, strides, NaN in rows
that nobody may see, and the ways a program calls it."""
import numpy as np
import pytest
import torch

from oracle import walks
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d

pytestmark = pytest.mark.gpu

LAYOUTS = [
    ([1], 1), ([1] * 5, 2), ([1] * 70, 1), ([32, 33, 31, 1, 2], 2), ([129, 40, 300, 7], 3), ([512], 1), ([513, 5], 2),
    ([700, 3, 3, 600], 2), ([40] * 30, 2), ([500, 20, 100, 530, 1], 4),
    # (at most 64 rows of documents of at most 32 tokens: the few-rows kernel)
    ([32, 31, 1], 2), ([3, 20, 30], 3), ([1] * 33, 2), ([16], 5),
]


def tensors(lens, heads, prefix, seed):
    S = sum(lens)
    return [W.rows(S, heads, seed + i) for i in range(3)] + [W.rows(prefix, heads, seed + 3 + i) for i in range(2)]


def oracle(p, t):
    q, k, v, kp, vp = (W.f64(x) for x in t)
    return walks.prefix_attention(q, k, v, kp, vp, p.cu, W.SCALE)


def status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


@pytest.mark.parametrize("lens,heads", LAYOUTS)
@pytest.mark.parametrize("prefix", [1, 127, 128, 300, 2430])
def test_forward_matches_the_oracle(lib, lens, heads, prefix):
    p = W.Prefix(lens, heads, prefix)
    t = tensors(lens, heads, prefix, 1)
    o, lse = p.forward(*t)
    W.ok(p.plan)
    W.check(o, lse, t[0], [t[1], t[3]], oracle(p, t), f"{lens} P={prefix}")


@pytest.mark.parametrize("lens,heads,prefix", [([1], 21, 20423), ([1] * 64, 21, 5033), ([2000, 2000], 8, 4096), ([31] * 40, 21, 640),
                                               ([300] * 12, 56, 1215), ([1] * 200, 21, 2430), ([1] * 128, 2, 1200),
                                               ([1] * 200, 1, 12000), ([32] * 9, 8, 300), ([30, 32, 31, 7, 1] * 5, 3, 5000),
                                               ([2] * 50, 2, 12000)])
def test_larger_batches(lib, lens, heads, prefix):
    p = W.Prefix(lens, heads, prefix)
    t = tensors(lens, heads, prefix, 10)
    o, lse = p.forward(*t)
    W.ok(p.plan)
    W.check(o, lse, t[0], [t[1], t[3]], oracle(p, t), f"{lens} P={prefix}")


def test_a_document_and_its_prefix_are_one_document(lib):
    # the dense forward over [prefix | document] gives the document's rows the same output
    P, L, heads = 640, 700, 2
    q, k, v = (W.rows(P + L, heads, 20 + i) for i in range(3))
    p = W.Prefix([L], heads, P)
    o, lse = p.forward(q[P:], k[P:], v[P:], k[:P], v[:P])
    o2, lse2 = W.outputs(P + L, heads)
    with H.Plan(docs_1d([P + L]), heads) as plan:
        H.h3attn_forward(plan.handle, W.flat(q), W.flat(k), W.flat(v), W.flat(o2), W.SCALE, lse2)
    assert (o.float() - o2[P:].float()).abs().max() <= 2.0 ** -6 and (lse - lse2[:, P:]).abs().max() <= 1e-4


@pytest.mark.parametrize("lens", [[1, 1, 1], [20, 40, 300], [700, 33, 600]])
def test_nan_in_other_documents_and_behind_the_prefix_reaches_nothing(lib, lens):
    heads, P = 2, 200
    p = W.Prefix(lens, heads, P)
    t = tensors(lens, heads, P, 30)
    want = oracle(p, t)
    buf = torch.full((2, P + 100, heads * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[0, :P], buf[1, :P] = W.flat(t[3]), W.flat(t[4])
    o, lse = p.forward(*t[:3], buf[0], buf[1])
    W.check(o, lse, t[0], [t[1], t[3]], want)
    for poison in (float("nan"), float("inf")):
        for d in range(len(lens)):
            a, b = p.cu[d], p.cu[d + 1]
            k2, v2 = t[1].clone(), t[2].clone()
            k2[a:b], v2[a:b] = poison, poison
            o2, lse2 = p.forward(t[0], k2, v2, t[3], t[4])
            keep = torch.ones(p.S, dtype=torch.bool, device="cuda")
            keep[a:b] = False
            assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[:, keep], lse[:, keep])
            assert not torch.isfinite(o2[a:b].float()).all()
    # and a poisoned query row stays alone
    q2 = t[0].clone()
    q2[0] = float("nan")
    o2, _ = p.forward(q2, *t[1:])
    assert torch.equal(o2[1:], o[1:])


@pytest.mark.parametrize("lens", [[1] * 9, [300, 40, 5], [1100]])
@pytest.mark.parametrize("spread,size", [(8.0, 1.0), (3.0, 2.0 ** 60), (0.0, 1.0)])
def test_wide_scores_and_large_values(lib, lens, spread, size):
    p = W.Prefix(lens, 2, 700)
    t = tensors(lens, 2, 700, 110)
    t[0] = (t[0].float() * spread).to(torch.bfloat16)
    t[2], t[4] = ((x.float() * size).to(torch.bfloat16) for x in (t[2], t[4]))
    o, lse = p.forward(*t)
    W.check(o, lse, t[0], [t[1], t[3]], oracle(p, t))


def test_strides_guards_and_no_lse(lib):
    lens, heads, P = [5, 333, 64], 2, 150
    p = W.Prefix(lens, heads, P)
    t = tensors(lens, heads, P, 40)
    o, _ = p.forward(*t)
    w = heads * 128
    own = [W.strided(x, w + 24) for x in t[:3]]
    pre = [W.strided(x, 3 * w) for x in t[3:]]
    out = torch.full((p.S + 3, w + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    H.h3attn_forward_prefix(p.plan.handle, *own, *pre, out[:p.S, :w], W.SCALE, None)
    assert torch.equal(out[:p.S, :w], W.flat(o))
    assert torch.all(out[p.S:] == 5.0) and torch.all(out[:, w:] == 5.0)


def test_offsets_past_32_bits(lib):
    # rows 2 MB apart: the last rows lie more than 2^32 bytes, and 2^31 elements, into the buffers
    stride, P, lens = 1 << 20, 2200, [1, 20, 2150]
    heads, S = 1, 2171
    p = W.Prefix(lens, heads, P)
    t = tensors(lens, heads, P, 50)
    o, lse = p.forward(*t)
    big = torch.empty(max(P, S), stride, dtype=torch.bfloat16, device="cuda")
    q, k, v = (big[:S, 256 * i:256 * i + 128] for i in range(3))
    kp, vp = (big[:P, 256 * i:256 * i + 128] for i in (3, 4))
    for dst, src in zip((q, k, v, kp, vp), t):
        dst.copy_(W.flat(src))
    o2, lse2 = p.forward(q, k, v, kp, vp)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    # selection and sparse forward over the same buffers
    s = W.Sparse(lens, heads, 256, 4)
    s.select(t[0], t[1], 4)
    idx = s.idx.clone()
    o, lse = s.forward(*t[:3])
    s.idx.fill_(-7)
    H.h3attn_block_select(s.plan.handle, q, k, 4, s.idx, s.cnt, keep_own=False)
    assert torch.equal(s.idx, idx)
    o2, lse2 = s.forward(q, k, v)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("lens", [[1, 20], [1] * 33])
def test_few_rows_offsets_past_32_bits(lib, lens):
    stride, P, heads = 1 << 20, 2200, 1
    p = W.Prefix(lens, heads, P)
    t = tensors(lens, heads, P, 51)
    o, lse = p.forward(*t)
    big = torch.empty(P, stride, dtype=torch.bfloat16, device="cuda")
    kp, vp = (big[:P, 256 * i:256 * i + 128] for i in (3, 4))
    for dst, src in zip((kp, vp), t[3:]):
        dst.copy_(W.flat(src))
    o2, lse2 = p.forward(*t[:3], kp, vp)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_captured_and_replayed_on_new_inputs(lib):
    lens, heads, P = [1, 600, 20, 50], 3, 900
    p = W.Prefix(lens, heads, P)
    t = tensors(lens, heads, P, 60)
    o, lse = W.outputs(p.S, heads)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        p.forward(*t, o, lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.forward(*t, o, lse)
    for seed in (70, 80):
        for x, y in zip(t, tensors(lens, heads, P, seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        W.ok(p.plan)
        W.check(o, lse, t[0], [t[1], t[3]], oracle(p, t))
        first = o.clone()
        o.fill_(0)
        p.forward(*t, o, lse)  # eager, the same bits
        assert torch.equal(o, first)


def test_both_lists_on_one_plan_and_the_dense_forward_unchanged(lib):
    lens, heads, P = [400, 260], 2, 300
    p = W.Prefix(lens, heads, P)
    t = tensors(lens, heads, P, 90)
    f = [W.flat(x) for x in t]
    o1, o2 = W.outputs(p.S, heads)[0], W.outputs(p.S, heads)[0]
    with H.Plan(docs_1d(lens), heads) as plain:
        H.h3attn_forward(plain.handle, *f[:3], W.flat(o1), W.SCALE)
        torch.cuda.synchronize()
    a = p.forward(*t)
    H.h3attn_plan_set_sparse(p.plan.handle, 512, 2)
    b = p.forward(*t)
    H.h3attn_forward(p.plan.handle, *f[:3], W.flat(o2), W.SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(o1, o2)


def test_refusals(lib):
    E = H.H3ATTN_EINVAL
    lens, heads, P = [300], 2, 100
    t = [W.flat(x) for x in tensors(lens, heads, P, 99)]
    o = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 300, device="cuda")
    with H.Plan(docs_1d(lens), heads) as plan:
        p = plan.handle
        fwd = lambda **kw: H.h3attn_forward_prefix(**{**dict(  # noqa: E731
            plan=p, q=t[0].data_ptr(), k=t[1].data_ptr(), v=t[2].data_ptr(), k_prefix=t[3].data_ptr(),
            v_prefix=t[4].data_ptr(), o=o.data_ptr(), softmax_scale=0.1, lse=lse.data_ptr(), qkv_row_stride=256,
            prefix_row_stride=256, o_row_stride=256), **kw})
        assert status(fwd) == E  # no prefix set
        for bad in (0, -1):
            assert status(lambda: H.h3attn_plan_set_prefix(p, bad)) == E
        H.h3attn_plan_set_prefix(p, P)
        assert status(lambda: H.h3attn_plan_set_prefix(p, P)) == E  # once per plan
        fwd()
        for kw in (dict(q=None), dict(k_prefix=None), dict(v_prefix=None), dict(k_prefix=t[3].data_ptr() + 8),
                   dict(prefix_row_stride=248), dict(prefix_row_stride=252), dict(qkv_row_stride=128), dict(o_row_stride=260),
                   dict(o=t[3].data_ptr()), dict(o=t[1].data_ptr()), dict(lse=t[4].data_ptr()), dict(lse=t[0].data_ptr()),
                   dict(lse=lse.data_ptr() + 2), dict(softmax_scale=-1.0), dict(softmax_scale=float("inf"))):
            assert status(lambda: fwd(**kw)) == E, kw
        with pytest.raises(ValueError):
            H.h3attn_forward_prefix(p, *t[:3], t[3], W.strided(t[4].view(100, 2, 128), 512), o, 0.1)
        # a prefix or batch that is too short, or not on the device
        for bad in (dict(k_prefix=t[3][:99], v_prefix=t[4][:99]), dict(q=t[0][:299]), dict(v_prefix=t[4].cpu())):
            with pytest.raises(ValueError):
                H.h3attn_forward_prefix(**{**dict(plan=p, q=t[0], k=t[1], v=t[2], k_prefix=t[3], v_prefix=t[4], o=o,
                                                  softmax_scale=0.1), **bad})
        torch.cuda.synchronize()

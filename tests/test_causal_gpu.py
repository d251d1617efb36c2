"""Causal attention with grouped heads on the GPU, against the fp64 oracle:
prompts from one token on, groups of every kind, strides, NaN in other
documents, and the ways a program calls it."""
import numpy as np
import pytest
import torch

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d, sample_rows

pytestmark = pytest.mark.gpu


class Causal:
    """A plan with a causal list and its calls."""

    def __init__(self, lens, heads, kv):
        self.lens, self.heads, self.kv = lens, heads, kv
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        self.S = int(self.cu[-1])
        self.plan = H.Plan(docs_1d(lens), heads)
        H.h3attn_plan_set_causal(self.plan.handle, kv)

    def inputs(self, seed):
        return [W.rows(self.S, h, seed + i) for i, h in enumerate((self.heads, self.kv, self.kv))]

    def forward(self, q, k, v, o=None, lse=None, with_lse=True, stream=None):
        o, lse = W.outputs(self.S, self.heads, o, lse)
        H.h3attn_forward_causal(self.plan.handle, q, k, v, o, W.SCALE, lse if with_lse else None, stream=stream)
        return o, lse

    def check(self, o, lse, t, rows=None, what=""):
        q, k, v = (W.f64(x) for x in t)
        want = serving.causal_attention(q, k, v, self.cu, W.SCALE, rows)
        at = slice(None) if rows is None else torch.from_numpy(rows).cuda()
        W.check(o[at], lse[:, at], t[0], [t[1]], want, what)


LAYOUTS = [[1], [1, 1, 1], [64, 80], [127, 128, 129], [17, 405, 1, 300], [511, 512, 513], [700, 2, 33]]


@pytest.mark.parametrize("lens", LAYOUTS)
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (4, 2), (6, 2), (4, 1), (10, 2), (6, 1), (7, 1), (16, 2), (9, 1), (11, 1), (16, 1),
                                      (17, 1), (34, 1)])
def test_forward_matches_the_oracle(lib, lens, heads, kv):
    c = Causal(lens, heads, kv)
    t = c.inputs(1)
    o, lse = c.forward(*t)
    W.ok(c.plan)
    c.check(o, lse, t, what=f"{lens} {heads}/{kv}")
    o2, _ = c.forward(*t, with_lse=False)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("lens,heads,kv", [([20423], 2, 1), ([5033], 28, 4), ([2430, 4096, 100], 21, 21), ([300] * 30, 32, 8),
                                           ([1400, 2576, 488, 3416], 48, 4), ([9000], 1, 1), ([1] * 300, 8, 2), ([3000], 2, 2)])
def test_longer_prompts(lib, lens, heads, kv):
    c = Causal(lens, heads, kv)
    t = c.inputs(10)
    o, lse = c.forward(*t)
    W.ok(c.plan)
    c.check(o, lse, t, sample_rows(c.cu, 24, 16), f"{lens}")
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


def test_the_last_row_is_the_dense_forward_s(lib):
    lens, heads = [1000, 77], 4
    c = Causal(lens, heads, heads)
    t = c.inputs(20)
    o, lse = c.forward(*t)
    o2, lse2 = W.outputs(c.S, heads)
    H.h3attn_forward(c.plan.handle, *(W.flat(x) for x in t), W.flat(o2), W.SCALE, lse2)
    last = [999, 1076]
    assert (o[last].float() - o2[last].float()).abs().max() <= 2.0 ** -6 and (lse[:, last] - lse2[:, last]).abs().max() <= 1e-4


@pytest.mark.parametrize("heads,kv", [(2, 2), (4, 1), (7, 1)])
def test_nan_elsewhere_reaches_nothing(lib, heads, kv):
    lens = [40, 300, 20, 700]
    c = Causal(lens, heads, kv)
    t = c.inputs(30)
    o, lse = c.forward(*t)
    for poison in (float("nan"), float("inf")):
        for d in range(len(lens)):
            a, b = int(c.cu[d]), int(c.cu[d + 1])
            k, v = t[1].clone(), t[2].clone()
            k[a:b], v[a:b] = poison, poison
            o2, lse2 = c.forward(t[0], k, v)
            keep = torch.ones(c.S, dtype=torch.bool, device="cuda")
            keep[a:b] = False
            assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[:, keep], lse[:, keep])
    # a later row's k reaches no earlier row, whatever it holds; its v none that is 512 before it
    k, v = t[1].clone(), t[2].clone()
    k[1059], v[1059] = float("nan"), float("nan")
    o2, lse2 = c.forward(t[0], k, t[2])
    assert torch.equal(o2[:1059], o[:1059]) and torch.equal(lse2[:, :1059], lse[:, :1059]) and not torch.isfinite(lse2[:, 1059]).any()
    o2, lse2 = c.forward(t[0], t[1], v)
    assert torch.equal(o2[:1059 - 511], o[:1059 - 511]) and torch.equal(lse2, lse)
    q = t[0].clone()
    q[100, 0] = float("nan")
    o2, _ = c.forward(q, *t[1:])
    o2[100, 0] = o[100, 0]
    assert torch.equal(o2, o)


@pytest.mark.parametrize("spread,size", [(8.0, 1.0), (3.0, 2.0 ** 60), (0.0, 1.0)])
def test_wide_scores_and_large_values(lib, spread, size):
    c = Causal([600, 90], 6, 2)
    t = c.inputs(40)
    t[0] = (t[0].float() * spread).to(torch.bfloat16)
    t[2] = (t[2].float() * size).to(torch.bfloat16)
    o, lse = c.forward(*t)
    c.check(o, lse, t)


@pytest.mark.parametrize("heads,kv", [(4, 2), (7, 1), (3, 3)])
def test_one_fused_buffer_strides_and_guards(lib, heads, kv):
    lens = [5, 333, 64]
    c = Causal(lens, heads, kv)
    t = c.inputs(50)
    o, lse = c.forward(*t)
    w = (heads + 2 * kv) * 128
    buf = torch.full((c.S + 3, w + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    cols = np.cumsum([0, heads * 128, kv * 128, kv * 128])
    parts = [buf[:c.S, a:b] for a, b in zip(cols[:-1], cols[1:])]
    for x, y in zip(parts, t):
        x.copy_(W.flat(y))
    for pad in (8, 16):  # 16-byte and 32-byte aligned rows
        out = torch.full((c.S + 3, heads * 128 + pad), 5.0, dtype=torch.bfloat16, device="cuda")
        H.h3attn_forward_causal(c.plan.handle, *parts, out[:c.S, :heads * 128], W.SCALE, None)
        assert torch.equal(out[:c.S, :heads * 128], W.flat(o))
        assert torch.all(out[c.S:] == 5.0) and torch.all(out[:, heads * 128:] == 5.0)


def test_offsets_past_32_bits(lib):
    stride, lens = 1 << 20, [20, 2150]
    c = Causal(lens, 2, 1)
    t = c.inputs(60)
    o, lse = c.forward(*t)
    big = torch.empty(c.S, stride, dtype=torch.bfloat16, device="cuda")
    far = [big[:, 512 * i:512 * i + 128 * h] for i, h in enumerate((2, 1, 1, 2))]
    for x, y in zip(far, t):
        x.copy_(W.flat(y))
    lse2 = torch.empty_like(lse)
    H.h3attn_forward_causal(c.plan.handle, *far, W.SCALE, lse2)
    assert torch.equal(far[3], W.flat(o)) and torch.equal(lse2, lse)


def test_captured_and_replayed_beside_the_other_calls(lib):
    # one plan with every list, its calls one after the other in one graph
    lens, heads, kv = [300, 1, 650], 4, 2
    c = Causal(lens, heads, kv)
    H.h3attn_plan_set_prefix(c.plan.handle, 100)
    t, kp = c.inputs(70), [W.rows(100, heads, 73), W.rows(100, heads, 74)]
    wide = [W.rows(c.S, heads, 75), W.rows(c.S, heads, 76)]
    o, lse = W.outputs(c.S, heads)
    o2, lse2 = W.outputs(c.S, heads)

    def both(stream=None):
        c.forward(*t, o, lse, stream=stream)
        H.h3attn_forward_prefix(c.plan.handle, t[0], *wide, *kp, o2, W.SCALE, lse2, stream=stream)

    side = torch.cuda.Stream()
    both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    for seed in (80, 90):
        for x, y in zip(t, c.inputs(seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        W.ok(c.plan)
        c.check(o, lse, t)
        got = [x.clone() for x in (o, lse, o2, lse2)]
        both()
        assert all(torch.equal(x, y) for x, y in zip(got, (o, lse, o2, lse2)))


def test_refusals(lib):
    E = H.H3ATTN_EINVAL

    def status(fn):
        with pytest.raises(H.H3AttnError) as e:
            fn()
        return e.value.status

    with H.Plan(docs_1d([300]), 4) as plan:
        p = plan.handle
        q, k, v = W.rows(300, 4, 1), W.rows(300, 2, 2), W.rows(300, 2, 3)
        o, lse = W.outputs(300, 4)
        fwd = lambda **kw: H.h3attn_forward_causal(**{**dict(  # noqa: E731
            plan=p, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), o=o.data_ptr(), softmax_scale=0.1, lse=lse.data_ptr(),
            q_row_stride=512, kv_row_stride=256, o_row_stride=512), **kw})
        assert status(fwd) == E  # no list
        for kv in (0, -2, 3, 8):
            assert status(lambda: H.h3attn_plan_set_causal(p, kv)) == E
        H.h3attn_plan_set_causal(p, 2)
        assert status(lambda: H.h3attn_plan_set_causal(p, 2)) == E  # once per plan
        fwd()
        for kw in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=q.data_ptr() + 8), dict(k=k.data_ptr() + 2),
                   dict(q_row_stride=256), dict(q_row_stride=516), dict(kv_row_stride=128), dict(kv_row_stride=252),
                   dict(o_row_stride=504), dict(o=q.data_ptr()), dict(o=k.data_ptr()), dict(o=v.data_ptr()),
                   dict(lse=q.data_ptr()), dict(lse=v.data_ptr()), dict(lse=o.data_ptr()), dict(lse=lse.data_ptr() + 2),
                   dict(softmax_scale=0.0), dict(softmax_scale=float("nan"))):
            assert status(lambda: fwd(**kw)) == E, kw
        good = dict(plan=p, q=q, k=k, v=v, o=o, softmax_scale=0.1, lse=lse)
        H.h3attn_forward_causal(**good)
        for kw in (dict(q=q[:299]), dict(q=q.float()), dict(k=k[:, :1]), dict(v=v.half()), dict(k=k.cpu()), dict(o=o[:, :3]),
                   dict(lse=lse[:3]), dict(lse=lse.double()), dict(v=W.strided(v, 512)), dict(k=k.transpose(0, 1))):
            with pytest.raises(ValueError):
                H.h3attn_forward_causal(**{**good, **kw})
        torch.cuda.synchronize()
        W.ok(plan)

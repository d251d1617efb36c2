"""Attention for trees of drafts over a paged cache on the GPU, against the fp64
oracle: contexts from none on, trees of 1 to 64, pages of many sizes and both
layouts, masks that leave nothing, NaN in every row that nobody may see, lengths
that grow under a captured graph, and what is reported and refused."""
import numpy as np
import pytest
import torch

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d

pytestmark = pytest.mark.gpu


class Tree:
    """A plan with a tree workspace, a cache full of NaN but for its sequences' rows, and its calls."""

    def __init__(self, ctx, drafts, heads, kv, page, head_major=False, seed=0, spare=0):
        self.ctx, self.drafts, self.heads, self.kv, self.page = list(ctx), list(drafts), heads, kv, page
        self.cu = np.concatenate([[0], np.cumsum(drafts)])
        self.S = int(self.cu[-1])
        self.plan = H.Plan(docs_1d(drafts), heads)
        H.h3attn_plan_set_tree(self.plan.handle, kv)
        need = [-(-(c + t + spare) // page) for c, t in zip(ctx, drafts)]
        self.pages = sum(need) + 3
        free = np.random.default_rng(seed).permutation(self.pages)
        self.table = np.full((len(ctx), max(need) + 2), -5, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = free[at:at + n]
            at += n
        shape = (self.pages, kv, page, 128) if head_major else (self.pages, page, kv, 128)
        full = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.kc, self.vc = (x.transpose(1, 2) if head_major else x for x in full)
        self.cache = H.Cache(self.kc, self.vc)
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_ctx = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        for b, (c, t) in enumerate(zip(ctx, drafts)):
            self.put(b, 0, W.rows(c + t, kv, seed + 100 + b), W.rows(c + t, kv, seed + 500 + b))
        self.q = W.rows(self.S, heads, seed + 1)

    def put(self, b, first, k, v):
        """Rows of sequence b from `first` on."""
        at = torch.from_numpy(serving.slots_of(self.table[b], first + len(k), self.page)[first:]).cuda()
        self.kc[at // self.page, at % self.page], self.vc[at // self.page, at % self.page] = k, v

    def forward(self, masks=None, q=None, o=None, lse=None, with_lse=True, stream=None, cache=None):
        o, lse = W.outputs(self.S, self.heads, o, lse)
        if masks is not None and not torch.is_tensor(masks):
            masks = words(masks)
        H.h3attn_forward_tree(self.plan.handle, self.q if q is None else q, cache or self.cache, self.d_table, self.d_ctx, o, W.SCALE,
                              lse if with_lse else None, tree_mask=masks, stream=stream)
        return o, lse

    def check(self, o, lse, masks=None, what=""):
        kc, vc = (W.f64(torch.nan_to_num(x.float())) for x in (self.kc, self.vc))
        ctx = self.d_ctx.tolist()
        want = serving.tree_attention(W.f64(self.q), kc, vc, self.table, ctx, self.cu, masks, W.SCALE)
        seen = [torch.nan_to_num(self.kc.float())]
        W.check(o, lse, self.q, seen, want, what)


def words(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")


def random_masks(drafts, seed):
    """Ancestors and self of random trees; a draft now and then that sees no draft at all."""
    rng, out = np.random.default_rng(seed), []
    for t in drafts:
        line = [1]
        for i in range(1, t):
            line.append(line[int(rng.integers(max(0, i - 9), i))] | 1 << i)
        if t > 3:
            line[2] = 0
        out += line
    return out


CASES = [
    ([0], [1], 1, 1, 8), ([1], [1], 4, 1, 16), ([127], [1], 8, 2, 16), ([128], [1], 8, 2, 64), ([0, 5, 300], [1, 1, 1], 7, 1, 32),
    ([0], [64], 4, 2, 16), ([100], [28], 2, 2, 128), ([64, 65, 63], [64, 63, 64], 8, 1, 16), ([1000, 3, 513], [5, 64, 17], 6, 2, 24),
    ([700], [33], 28, 4, 256), ([2000, 0, 129, 900], [16, 16, 1, 3], 12, 4, 48), ([333] * 40, [1] * 40, 16, 2, 16),
    ([40] * 200, [2] * 200, 3, 3, 8), ([(37 * i * i) % 700 for i in range(160)], [1 + i % 5 for i in range(160)], 4, 2, 16),
    ([0] * 153, [1] * 153, 2, 1, 8), ([3000] + [0, 130, 127, 1] * 40, [1] * 161, 5, 1, 32), ([777], [9], 71, 1, 64), ([500], [10], 128, 1, 16), ([300, 20], [7, 50], 160, 1, 8),
]


@pytest.mark.parametrize("ctx,drafts,heads,kv,page", CASES)
@pytest.mark.parametrize("head_major", [False, True])
def test_forward_matches_the_oracle(lib, ctx, drafts, heads, kv, page, head_major):
    t = Tree(ctx, drafts, heads, kv, page, head_major)
    for masks in (None, random_masks(drafts, 3)):
        o, lse = t.forward(masks)
        W.ok(t.plan)
        t.check(o, lse, masks, f"{ctx[:4]} {drafts[:4]}")
    o2, _ = t.forward(masks, with_lse=False)
    assert torch.equal(o2, o)


@pytest.mark.parametrize("ctx,drafts,heads,kv,page", [([20423], [1], 8, 1, 16), ([20423, 9000], [64, 64], 16, 2, 128),
                                                      ([5033] * 32, [1] * 32, 8, 2, 16), ([3000, 100, 7000, 0, 1], [16] * 5, 28, 4, 64),
                                                      ([12000], [64], 64, 8, 64), ([600] * 64, [4] * 64, 32, 8, 32),
                                                      # one long sequence among many short ones: ranges of one
                                                      # piece beside ranges of many, in one block
                                                      ([7] * 40 + [9000] + [7] * 260, [1] * 301, 2, 1, 16),
                                                      # items of one query tile and of two, of one key tile and of many
                                                      ([300, 5, 900, 40, 0] * 40, [64, 1, 16, 2, 17] * 40, 8, 1, 16)])
def test_longer_contexts(lib, ctx, drafts, heads, kv, page):
    t = Tree(ctx, drafts, heads, kv, page)
    masks = random_masks(drafts, 5)
    o, lse = t.forward(masks)
    W.ok(t.plan)
    t.check(o, lse, masks)
    for _ in range(3):  # the same bits every time
        o2, lse2 = t.forward(masks)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_every_length_of_a_few_tiles(lib):
    # tile and page ends fall everywhere; one plan, lengths on the device
    t = Tree([400] * 2, [1, 6], 4, 2, 24)
    for n in list(range(0, 140)) + [255, 256, 257, 383, 400]:
        t.d_ctx.copy_(torch.tensor([n, max(0, n - 3)], dtype=torch.int32))
        # (the drafts' rows are those that lie behind the context)
        o, lse = t.forward()
        t.check(o, lse, what=f"{n}")
    W.ok(t.plan)


def test_rows_that_see_nothing(lib):
    t = Tree([0, 0, 200], [3, 1, 2], 4, 1, 16)
    masks = [0, 2, 0b101, 0, 0, 3]
    o, lse = t.forward(masks)
    W.ok(t.plan)
    t.check(o, lse, masks)
    for row in (0, 3):
        assert not o[row].float().any() and torch.isneginf(lse[:, row]).all()
    # bits past the tree are no drafts
    o2, lse2 = t.forward([m | 0xF0 << 56 | 1 << 40 for m in masks])
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("spread,size", [(8.0, 1.0), (3.0, 2.0 ** 60), (0.0, 1.0)])
def test_wide_scores_and_large_values(lib, spread, size):
    t = Tree([900, 50], [5, 64], 8, 2, 16)
    t.q = (t.q.float() * spread).to(torch.bfloat16)
    t.vc.copy_((t.vc.float() * size).to(torch.bfloat16))
    o, lse = t.forward()
    t.check(o, lse)


@pytest.mark.parametrize("steps", [[0, 24] * 8, [24 * i for i in range(8)], [0, 0, 0, 48, 0, 96, 24, 120]])
@pytest.mark.parametrize("ctx,drafts", [([496], [16]), ([448, 300, 60] * 60, [1] * 180)])
def test_scores_that_step_up_between_halves_of_a_tile(lib, steps, ctx, drafts):
    # every 64 keys the scores of even heads step by 34 (49 in powers of two) a 24, those of odd heads fall; the
    # references move inside a tile, in some rows of a warp only, and what was summed before them counts 2^-49 or 0
    t = Tree(ctx, drafts, 8, 2, 16)
    t.q[:, 0::2, 0], t.q[:, 1::2, 0] = 16.0, -16.0
    for b, (c, d) in enumerate(zip(ctx, drafts)):
        k, v = W.rows(c + d, 2, 100 + b), W.rows(c + d, 2, 500 + b)
        k[:, :, 0] = torch.tensor([float(steps[i // 64]) for i in range(c + d)], device="cuda")[:, None]
        t.put(b, 0, k, v)
    t.check(*t.forward(), what=steps)


@pytest.mark.parametrize("ctx,drafts,heads,kv", [
    ([(53 * i * i) % 1400 for i in range(140)], [1 + i % 3 for i in range(140)], 4, 1),   # a block to an item and a bit: ranges, one tile
    ([(53 * i * i) % 1400 for i in range(140)], [9 + i % 8 for i in range(140)], 16, 1),   # and two tiles
    ([(53 * i * i) % 1400 for i in range(70)], [40] * 70, 32, 2),   # more items than blocks, of two tiles and of one
    ([700 + 9 * i for i in range(100)], [1] * 100, 8, 1),           # pieces, several sequences to a lane
    ([1200] * 33, [2] * 33, 8, 4)])                                 # pieces above the even share
def test_every_way_of_cutting_the_work(lib, ctx, drafts, heads, kv):
    t = Tree(ctx, drafts, heads, kv, 32)
    first = t.forward()
    t.check(*first)
    again = t.forward()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_table_for_very_long_sequences(lib):
    # 2^28 rows and more to a sequence's table: the lengths are added up another way
    ctx, page = [4000, 130, 1], 1 << 16
    t = Tree(ctx, [3, 1, 64], 8, 1, page)
    t.check(*t.forward())
    wide = torch.full((3, (1 << 28) // page + 1), -9, dtype=torch.int32, device="cuda")
    wide[:, :t.table.shape[1]] = t.d_table
    t.d_table = wide
    o, lse = t.forward()
    t.table = wide.cpu().numpy()
    t.check(o, lse)


def test_stacked_layers_strides_and_guards(lib):
    # a cache whose layers, k and v share one buffer; q out of a fused one; o with guards
    ctx, drafts, heads, kv, page = [300, 40], [6, 1], 6, 2, 16
    t = Tree(ctx, drafts, heads, kv, page)
    o, lse = t.forward()
    buf = torch.full((t.pages, 3, 2, page, kv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, 1, 0], buf[:, 1, 1] = t.kc, t.vc
    cache = H.Cache(buf[:, 1, 0], buf[:, 1, 1])
    wide = W.strided(t.q, (heads + 2 * kv) * 128)
    out = torch.full((t.S + 2, heads * 128 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    H.h3attn_forward_tree(t.plan.handle, wide, cache, t.d_table, t.d_ctx, out[:t.S, :heads * 128], W.SCALE)
    assert torch.equal(out[:t.S, :heads * 128], W.flat(o))
    assert torch.all(out[t.S:] == 5.0) and torch.all(out[:, heads * 128:] == 5.0)


def test_a_cache_past_32_bits(lib):
    ctx, drafts, kv, page = [700], [3], 1, 8
    t = Tree(ctx, drafts, 2, kv, page)
    o, lse = t.forward()
    big = torch.empty(t.pages, 1 << 25, dtype=torch.bfloat16, device="cuda")  # 64 MB a page
    k, v = (big[:, i * 4096:i * 4096 + 1024].view(t.pages, page, 1, 128) for i in range(2))
    k.copy_(t.kc), v.copy_(t.vc)
    o2, lse2 = t.forward(cache=H.Cache(k, v))
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_a_graph_serves_sequences_as_they_grow(lib):
    # the whole step captured: rotary and store, attention, and the accepted drafts move up; lengths, slots,
    # masks and tables change between replays, the graph does not
    ctx, drafts, heads, kv, page = [250, 0, 126], [4, 4, 1], 8, 2, 16
    t = Tree(ctx, drafts, heads, kv, page, spare=40)
    rope = H.h3attn_rope_init(128, 1e4)
    S = t.S
    x = [W.rows(S, h, 900 + i) for i, h in enumerate((heads, kv, kv))]
    pos, slots = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
    src, dst = (torch.full((3, 4), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    masks = words(random_masks(drafts, 1))
    o, lse = W.outputs(S, heads)

    def step(stream=None):
        H.h3attn_rotary_store(rope, pos, x[0], t.q, x[1], x[2], t.cache, slots, stream=stream)
        H.h3attn_forward_tree(t.plan.handle, t.q, t.cache, t.d_table, t.d_ctx, o, W.SCALE, lse, tree_mask=masks, stream=stream)
        H.h3attn_cache_move(t.cache, src, dst, stream=stream)

    side = torch.cuda.Stream()
    slots.fill_(-1)
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    n = list(ctx)
    rng = np.random.default_rng(2)
    for it in range(6):
        tree = random_masks(drafts, 10 + it)
        at = [serving.slots_of(t.table[b], n[b] + drafts[b], page)[n[b]:] for b in range(3)]
        accept = [sorted(rng.choice(range(1, d), int(rng.integers(0, d)), replace=False).tolist()) if d > 1 else [] for d in drafts]
        accept = [[0] + a for a in accept]
        src.fill_(-1), dst.fill_(-1)
        for b in range(3):
            for i, a in enumerate(accept[b]):
                src[b, i], dst[b, i] = int(at[b][a]), int(at[b][i])
        slots.copy_(torch.from_numpy(np.concatenate(at).astype(np.int32)))
        pos.copy_(torch.tensor([n[b] + bin(tree[t.cu[b] + i]).count("1") - 1 if tree[t.cu[b] + i] else n[b] for b in range(3)
                                for i in range(drafts[b])], dtype=torch.int32))
        t.d_ctx.copy_(torch.tensor(n, dtype=torch.int32))
        masks.copy_(words(tree))
        for i, y in enumerate(x):
            y.copy_(W.rows(S, y.shape[1], 1000 + 10 * it + i))
        graph.replay()
        torch.cuda.synchronize()
        W.ok(t.plan)
        # the stored rows, the attention over them (before the move), and the moved rows
        k2 = torch.empty_like(x[1])
        H.h3attn_rotary(rope, pos, None, None, x[1], k2)
        flat = t.kc.reshape(-1, kv, 128)
        for b in range(3):
            for i, a in enumerate(accept[b]):
                assert torch.equal(flat[at[b][i]], k2[t.cu[b] + a])
            t.put(b, n[b], k2[t.cu[b]:t.cu[b + 1]], x[2][t.cu[b]:t.cu[b + 1]])
        t.check(o, lse, tree, f"step {it}")
        H.h3attn_cache_move(t.cache, src, dst)
        n = [c + len(a) for c, a in zip(n, accept)]


def test_every_list_on_one_plan_and_two_plans_at_once(lib):
    # trees beside the causal and prefix forwards of the same plan; and two plans on two streams
    ctx, drafts, heads, kv = [3000, 10], [30, 3], 4, 2
    a, b = Tree(ctx, drafts, heads, kv, 16, seed=1), Tree([500, 2500], drafts, heads, kv, 64, seed=2)
    H.h3attn_plan_set_causal(a.plan.handle, kv)
    H.h3attn_plan_set_prefix(a.plan.handle, 50)
    ref = [a.forward(), b.forward()]
    k, v = W.rows(a.S, kv, 5), W.rows(a.S, kv, 6)
    o, lse = W.outputs(a.S, heads)
    H.h3attn_forward_causal(a.plan.handle, a.q, k, v, o, W.SCALE, lse)
    want = serving.causal_attention(*(W.f64(x) for x in (a.q, k, v)), a.cu, W.SCALE)
    W.check(o, lse, a.q, [k], want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [W.outputs(t.S, heads) for t in (a, b)]
        torch.cuda.synchronize()
        for t, s, (o, lse) in zip((a, b), streams, outs):
            t.forward(o=o, lse=lse, stream=s)
        torch.cuda.synchronize()
        for (o, lse), (o2, lse2) in zip(outs, ref):
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_bad_pages_and_lengths_are_reported(lib):
    t = Tree([200, 100], [2, 2], 4, 2, 16)
    o, lse = t.forward()
    W.ok(t.plan)

    def reported():
        with pytest.raises(H.H3AttnError) as e:
            W.ok(t.plan)
        return e.value.status == H.H3ATTN_EINVAL and "page" in str(e.value)

    # a page outside the cache is rows of zeros: the other sequence is as it was
    for bad in (t.pages, -1, 2 ** 31 - 1, -2 ** 31):
        good = int(t.d_table[0, 3])
        t.d_table[0, 3] = bad
        o2, lse2 = t.forward()
        assert reported()
        t.d_table[0, 3] = good
        assert torch.equal(o2[2:], o[2:]) and torch.equal(lse2[:, 2:], lse[:, 2:])
        kc, vc = t.kc.clone(), t.vc.clone()
        t.kc[good], t.vc[good] = 0, 0
        t.check(o2, lse2)
        t.kc.copy_(kc), t.vc.copy_(vc)
        W.ok(t.plan)  # (the word was cleared)
    # a negative length is none; one past the table's is the table's
    t.d_ctx[1] = -7
    o2, lse2 = t.forward()
    assert reported() and torch.equal(o2[:2], o[:2])
    t.d_ctx[1] = 0
    o3, lse3 = t.forward()
    assert torch.equal(o3, o2) and torch.equal(lse3, lse2)
    W.ok(t.plan)
    most = t.d_table.shape[1] * t.page - 2
    t.d_table.clamp_(min=0)
    t.kc.nan_to_num_(0.0), t.vc.nan_to_num_(0.0)
    for n in (most + 1, 2 ** 31 - 1):
        t.d_ctx[1] = n
        o2, lse2 = t.forward()
        assert reported() and torch.equal(o2[:2], o[:2])
        t.d_ctx[1] = most
        o3, lse3 = t.forward()
        assert torch.equal(o3, o2) and torch.equal(lse3, lse2)
        W.ok(t.plan)


def test_refusals(lib):
    E, U = H.H3ATTN_EINVAL, H.H3ATTN_EUNSUPPORTED

    def status(fn):
        with pytest.raises(H.H3AttnError) as e:
            fn()
        return e.value.status

    with H.Plan(docs_1d([65]), 4) as plan:
        assert status(lambda: H.h3attn_plan_set_tree(plan.handle, 4)) == U
    with H.Plan(docs_1d([1] * 4097), 1) as plan:
        assert status(lambda: H.h3attn_plan_set_tree(plan.handle, 1)) == U
    t = Tree([20, 30], [3, 4], 4, 2, 16)
    p = t.plan.handle
    assert status(lambda: H.h3attn_plan_set_tree(p, 2)) == E  # once per plan
    with H.Plan(docs_1d([3, 4]), 4) as other:
        for kv in (0, -1, 3, 8):
            assert status(lambda: H.h3attn_plan_set_tree(other.handle, kv)) == E
        assert status(lambda: H.h3attn_forward_tree(other.handle, t.q, t.cache, t.d_table, t.d_ctx, t.q.clone(), 0.1, q_row_stride=512,
                                                    o_row_stride=512)) == E  # no workspace
    o, lse = W.outputs(t.S, 4)
    masks = words([1] * 7)
    good = dict(plan=p, q=t.q, cache=t.cache, page_table=t.d_table, ctx_lens=t.d_ctx, o=o, softmax_scale=0.1, lse=lse, tree_mask=masks)
    H.h3attn_forward_tree(**good)
    W.ok(t.plan)
    for kw in (dict(q=None, q_row_stride=512), dict(o=None, o_row_stride=512), dict(q=t.q.data_ptr() + 8, q_row_stride=512),
               dict(q=t.q.data_ptr(), q_row_stride=256), dict(o=t.q), dict(o=t.kc.view(-1, 4, 128)[:7]), dict(softmax_scale=-1.0),
               dict(o=t.vc.data_ptr() - 1024, o_row_stride=512), dict(lse=o.data_ptr()), dict(lse=t.kc.data_ptr()),
               dict(lse=t.d_table.data_ptr()), dict(o=t.d_ctx.data_ptr() // 16 * 16, o_row_stride=512), dict(lse=masks.data_ptr()),
               dict(lse=t.q.data_ptr()), dict(tree_mask=masks.data_ptr() + 4), dict(cache=H.Cache(t.kc[:, :, :1], t.vc[:, :, :1])),
               dict(page_table=torch.empty(2, 0, dtype=torch.int32, device="cuda"))):
        assert status(lambda: H.h3attn_forward_tree(**{**good, **kw})) == E, kw
    odd = [torch.zeros(8, 12, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert status(lambda: H.h3attn_forward_tree(**{**good, "cache": H.Cache(*odd)})) == U
    for kw in (dict(q=t.q[:6]), dict(q=t.q.float()), dict(o=o[:, :3]), dict(lse=lse[:3]), dict(page_table=t.d_table[:1]),
               dict(page_table=t.d_table.long()), dict(page_table=t.d_table[:, ::2]), dict(page_table=t.d_table.cpu()), dict(page_table=t.d_table[0]),
               dict(ctx_lens=t.d_ctx[:1]), dict(ctx_lens=t.d_ctx.long()), dict(ctx_lens=t.d_ctx.cpu()), dict(tree_mask=masks[:6]),
               dict(tree_mask=masks.int()), dict(tree_mask=masks.cpu())):
        with pytest.raises(ValueError):
            H.h3attn_forward_tree(**{**good, **kw})
    torch.cuda.synchronize()
    W.ok(t.plan)

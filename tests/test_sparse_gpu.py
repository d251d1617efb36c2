"""Block selection and the block-sparse forward on the GPU, against the fp64
oracle: layouts from one token on, lists of every kind (selected, shuffled,
repeated, empty, out of range), strides, NaN in keys that nobody may see, and
the ways a program calls them (captured, on other streams, without lse)."""
import numpy as np
import pytest
import torch

from oracle import walks
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d

pytestmark = pytest.mark.gpu

LAYOUTS = [
    ([1], 1), ([127], 1), ([128, 1, 129], 2), ([64, 80], 2), ([255, 256, 257], 3), ([511, 513, 2], 2),
    ([1500, 7, 700], 5), ([2177], 4),
]


def status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


# ---------------------------------------------------------------- selection ----

@pytest.mark.parametrize("lens,heads", LAYOUTS + [([4608, 384], 2), ([12800], 1)])
@pytest.mark.parametrize("q_block", [256, 512])
@pytest.mark.parametrize("keep,keep_own", [(1, False), (3, True), (9, False)])
def test_selection_is_the_oracles(lib, lens, heads, q_block, keep, keep_own):
    s = W.Sparse(lens, heads, q_block, keep + 2)
    q, k = W.rows(s.S, heads, 1), W.rows(s.S, heads, 2)
    idx, cnt = s.select(q, k, keep, keep_own)
    want = walks.select(W.f64(q), W.f64(k), s.cu, q_block, keep, keep_own, width=keep + 2)
    assert np.array_equal(cnt, want[1])
    assert np.array_equal(idx, want[0])


def test_selection_breaks_ties_by_the_lower_tile(lib):
    # equal key tiles score equally; zero queries score zero everywhere
    s = W.Sparse([1408], 2, 512, 11)
    q, k = W.rows(1408, 2, 3), W.rows(128, 2, 4).repeat(11, 1, 1)
    q[512:1024] = 0
    for keep in (1, 5, 11):
        idx, cnt = s.select(q, k, keep)
        assert np.all(cnt == keep)
        assert np.all(idx[:, :, :keep] == np.arange(keep)) and np.all(idx[:, :, keep:] == -1)
    # keep_own: the block's own four tiles first, the rest of the budget from the lowest
    idx, _ = s.select(q, k, 6, keep_own=True)
    assert idx[0, 1, :6].tolist() == [0, 1, 4, 5, 6, 7] and idx[0, 2, :6].tolist() == [0, 1, 2, 8, 9, 10]
    idx, _ = s.select(q, k, 2, keep_own=True)
    assert idx[0, 1, :2].tolist() == [4, 5]


@pytest.mark.parametrize("scale_k", [1.0, 2.0 ** -20, 2.0 ** 20])
def test_selection_resolves_scores_that_fp32_would_not(lib, scale_k):
    # eight tiles whose scores are M + small - M + what they share, the small terms
    # 2^-26 of M: lost in an fp32 sum
    k = W.rows(128, 1, 5).repeat(8, 1, 1)
    k[:, :, 0], k[:, :, 4] = 2.0 ** 14, -(2.0 ** 14)
    for t in range(8):
        k[128 * t:128 * t + 128, 0, 2] = 2.0 ** -12 * ((5 * t) % 8)
    k = (k.float() * scale_k).to(torch.bfloat16)
    q = W.rows(1024, 1, 6)
    q[:, :, 0], q[:, :, 2], q[:, :, 4] = 1.0, 1.0, 1.0
    s = W.Sparse([1024], 1, 512, 3)
    idx, cnt = s.select(q, k, 3)
    want = walks.select(W.f64(q), W.f64(k), s.cu, 512, 3, False)
    assert np.array_equal(idx, want[0]) and np.array_equal(cnt, want[1])
    assert idx[0, 0].tolist() == [1, 3, 6]  # (5 t) % 8 = 5, 7, 6: the largest three


def test_selection_ranks_nan_last_and_infinities_in_order(lib):
    s = W.Sparse([768], 1, 512, 6)
    q, k = W.rows(768, 1, 7).abs(), W.rows(768, 1, 8)
    k[130, 0, 3] = float("nan")
    k[260, 0, 3] = float("inf")
    k[400, 0, 3] = float("-inf")
    idx, _ = s.select(q, k, 1)
    assert np.all(idx[:, :, 0] == 2)
    idx, _ = s.select(q, k, 4)
    assert np.all(idx[:, :, :4] == [0, 2, 4, 5])
    idx, _ = s.select(q, k, 5)
    assert np.all(idx[:, :, :5] == [0, 2, 3, 4, 5])


def test_selection_of_a_long_document(lib):
    # 300 tiles: several chunks of the scoring loop, more than one group of blocks
    n = 300 * 128 - 5
    s = W.Sparse([n], 1, 512, 64)
    q, k = W.rows(n, 1, 9), W.rows(n, 1, 10)
    idx, cnt = s.select(q, k, 64, keep_own=True)
    want = walks.select(W.f64(q), W.f64(k), s.cu, 512, 64, True)
    assert np.array_equal(idx, want[0]) and np.array_equal(cnt, want[1])


def test_selection_reads_a_fused_buffer_and_only_its_rows(lib):
    lens, heads = [300, 77], 2
    s = W.Sparse(lens, heads, 256, 2)
    q, k = W.rows(s.S, heads, 11), W.rows(s.S, heads, 12)
    buf = torch.full((s.S, 3 * heads * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :heads * 128] = W.flat(q)
    buf[:, heads * 128:2 * heads * 128] = W.flat(k)
    H.h3attn_block_select(s.plan.handle, buf[:, :heads * 128], buf[:, heads * 128:2 * heads * 128], 2, s.idx, s.cnt,
                          keep_own=False)
    got = s.idx.cpu().numpy().copy()
    assert np.array_equal(got, s.select(q, k, 2)[0])


# ------------------------------------------------------------------ forward ----

def random_lists(s, rng, kind):
    idx = np.full((s.heads, s.nq, s.max_blocks), -1, dtype=np.int32)
    cnt = np.zeros((s.heads, s.nq), dtype=np.int32)
    for i, (_, _, a, b) in enumerate(walks.blocks(s.cu, s.q_block)):
        tiles = -(-(b - a) // 128)
        for h in range(s.heads):
            if kind == "shuffled":   # any number of tiles, none among them, in any order
                n = int(rng.integers(0, min(tiles, s.max_blocks) + 1))
                pick = rng.permutation(tiles)[:n]
            elif kind == "repeated":  # the same tiles more than once
                n = int(rng.integers(1, s.max_blocks + 1))
                pick = rng.integers(0, tiles, n)
            elif kind == "last":      # the ragged tile alone
                pick = np.array([tiles - 1])
            else:                     # every tile
                pick = np.arange(min(tiles, s.max_blocks))
            idx[h, i, :len(pick)] = pick
            cnt[h, i] = len(pick)
    return idx, cnt


@pytest.mark.parametrize("lens,heads", LAYOUTS)
@pytest.mark.parametrize("q_block", [256, 512])
@pytest.mark.parametrize("kind", ["shuffled", "repeated", "last", "all"])
def test_forward_matches_the_oracle(lib, lens, heads, q_block, kind):
    s = W.Sparse(lens, heads, q_block, 18 if kind == "all" else 5)
    q, k, v = (W.rows(s.S, heads, 20 + i) for i in range(3))
    idx, cnt = random_lists(s, np.random.default_rng(1), kind)
    s.lists(idx, cnt)
    o, lse = s.forward(q, k, v)
    W.ok(s.plan)
    want = walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, q_block, idx, cnt, W.SCALE)
    W.check(o, lse, q, [k], want, f"{lens} {kind}")


def test_all_tiles_agree_with_the_dense_forward(lib):
    lens, heads = [1500, 700], 3
    s = W.Sparse(lens, heads, 512, 12)
    q, k, v = (W.rows(s.S, heads, 30 + i) for i in range(3))
    s.lists(*random_lists(s, None, "all"))
    o, lse = s.forward(q, k, v)
    o2, lse2 = W.outputs(s.S, heads)
    H.h3attn_forward(s.plan.handle, W.flat(q), W.flat(k), W.flat(v), W.flat(o2), W.SCALE, lse2)
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -6 and (lse - lse2).abs().max() <= 1e-4


@pytest.mark.parametrize("q_block", [256, 512])
def test_empty_lists_and_negative_or_large_counts(lib, q_block):
    s = W.Sparse([700, 40], 2, q_block, 3)
    q, k, v = (W.rows(s.S, 2, 40 + i) for i in range(3))
    idx, cnt = random_lists(s, None, "all")
    cnt[0, 0], cnt[1, -1] = 0, -3
    s.lists(idx, cnt)
    o, lse = s.forward(q, k, v)
    want = walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, q_block, idx, np.maximum(cnt, 0), W.SCALE)
    W.check(o, lse, q, [k], want)
    assert torch.all(o[:min(q_block, 700), 0] == 0) and torch.all(lse[1, -40:] == -np.inf)
    cnt[0, 0] = 1 << 30  # clamped to max_blocks
    s.lists(idx, cnt)
    o, lse = s.forward(q, k, v)
    cnt[0, 0] = 3
    want = walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, q_block, idx, np.maximum(cnt, 0), W.SCALE)
    W.check(o, lse, q, [k], want)
    W.ok(s.plan)
    # nothing listed anywhere, in pieces too: zeros everywhere
    s.lists(idx, np.zeros_like(cnt))
    o, lse = s.forward(q, k, v)
    assert torch.all(o == 0) and torch.all(lse == -np.inf)


def test_tiles_outside_the_document_are_skipped_and_reported(lib):
    s = W.Sparse([300, 500], 1, 512, 4)
    q, k, v = (W.rows(s.S, 1, 50 + i) for i in range(3))
    idx = np.array([[[0, 3, 2, -1], [4, 3, 1 << 30, 0]]], dtype=np.int32)
    s.lists(idx, np.full((1, 2), 4, dtype=np.int32))
    o, lse = s.forward(q, k, v)
    assert status(lambda: W.ok(s.plan)) == H.H3ATTN_EINVAL
    W.ok(s.plan)  # the word is cleared
    idx2 = np.array([[[0, 2, -1, -1], [3, 0, -1, -1]]], dtype=np.int32)
    want = walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, 512, idx2, np.full((1, 2), 2), W.SCALE)
    W.check(o, lse, q, [k], want)


def test_nan_in_unlisted_keys_reaches_nothing(lib):
    # rows of other documents behind a ragged end, and whole unlisted tiles
    lens = [300, 70, 513]
    s = W.Sparse(lens, 2, 256, 3)
    q, k, v = (W.rows(s.S, 2, 60 + i) for i in range(3))
    idx, cnt = random_lists(s, None, "last")
    s.lists(idx, cnt)
    want = walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, 256, idx, cnt, W.SCALE)
    seen = np.zeros(s.S, dtype=bool)
    for a, b in zip(s.cu[:-1], s.cu[1:]):
        seen[a + (b - a - 1) // 128 * 128:b] = True
    bad = torch.from_numpy(~seen).cuda()
    for poison in (float("nan"), float("inf"), float("-inf")):
        k2, v2 = k.clone(), v.clone()
        k2[bad], v2[bad] = poison, poison
        o, lse = s.forward(q, k2, v2)
        W.check(o, lse, q, [k], want, str(poison))
    # the next document's rows in a ragged tile: poison one document, read another
    for d in range(3):
        k2, v2 = k.clone(), v.clone()
        k2[s.cu[d]:s.cu[d + 1]] = float("nan")
        v2[s.cu[d]:s.cu[d + 1]] = float("nan")
        o, _ = s.forward(q, k2, v2)
        for e in range(3):
            fine = torch.isfinite(o[s.cu[e]:s.cu[e + 1]]).all()
            assert bool(fine) == (e != d)


@pytest.mark.parametrize("q_block,max_blocks", [(256, 6), (512, 6), (512, 14)])
@pytest.mark.parametrize("spread,size", [(8.0, 1.0), (3.0, 2.0 ** 60), (0.0, 1.0)])
def test_wide_scores_and_large_values(lib, q_block, max_blocks, spread, size):
    # scores spread over hundreds of log2 units (maxima that grow past the rescale
    # threshold), over tens with large values (no rescale), and all equal
    s = W.Sparse([1700, 300], 2, q_block, max_blocks)
    q, k = W.rows(s.S, 2, 130, spread), W.rows(s.S, 2, 131)
    v = W.rows(s.S, 2, 132, size)
    idx, cnt = random_lists(s, np.random.default_rng(3), "shuffled")
    s.lists(idx, cnt)
    o, lse = s.forward(q, k, v)
    W.check(o, lse, q, [k], walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, q_block, idx, cnt, W.SCALE))


def test_strides_guards_and_no_lse(lib):
    lens, heads = [333, 64], 2
    s = W.Sparse(lens, heads, 256, 3)
    q, k, v = (W.rows(s.S, heads, 70 + i) for i in range(3))
    idx, cnt = random_lists(s, None, "all")
    s.lists(idx, cnt)
    o, lse = s.forward(q, k, v)
    wide = [W.strided(t, heads * 128 + 24) for t in (q, k, v)]
    out = torch.full((s.S + 3, heads * 128 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    H.h3attn_forward_sparse(s.plan.handle, *wide, s.idx, s.cnt, out[:s.S, :heads * 128], W.SCALE, None)
    assert torch.equal(out[:s.S, :heads * 128], W.flat(o))
    assert torch.all(out[s.S:] == 5.0) and torch.all(out[:, heads * 128:] == 5.0)


def test_select_and_forward_captured_and_replayed_on_new_inputs(lib):
    lens, heads = [1300, 260], 3
    s = W.Sparse(lens, heads, 512, 4)
    q, k, v = (W.rows(s.S, heads, 80 + i) for i in range(3))
    o, lse = W.outputs(s.S, heads)

    def step():
        H.h3attn_block_select(s.plan.handle, W.flat(q), W.flat(k), 4, s.idx, s.cnt, keep_own=True)
        s.forward(q, k, v, o, lse)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (90, 95):
        for i, t in enumerate((q, k, v)):
            t.copy_(W.rows(s.S, heads, seed + i))
        graph.replay()
        torch.cuda.synchronize()
        W.ok(s.plan)
        idx, cnt = walks.select(W.f64(q), W.f64(k), s.cu, 512, 4, True)
        assert np.array_equal(s.idx.cpu().numpy(), idx)
        W.check(o, lse, q, [k], walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, 512, idx, cnt, W.SCALE))
        first = o.clone()
        o.fill_(0)
        step()  # eager, the same bits
        assert torch.equal(o, first)


def test_two_plans_on_two_streams(lib):
    runs = []
    for seed, lens in ((100, [900, 33]), (110, [2048])):
        s = W.Sparse(lens, 2, 256, 4)
        t = [W.rows(s.S, 2, seed + i) for i in range(3)]
        s.select(t[0], t[1], 4)
        runs.append((s, t, s.forward(*t), torch.cuda.Stream(), W.outputs(s.S, 2)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, t, _, stream, out in runs:
            s.forward(*t, *out, stream=stream)
    torch.cuda.synchronize()
    for s, _, want, _, out in runs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_prologue_selection_and_sparse_forward_together(lib):
    # a block of the request's loop: raw q and k, 3D positions, sparse attention
    from tests.gpu_cases import random_tensors
    from synth.device import bf16_to_torch
    docs = [[(2, 15, 27, (0.0, 0.0, 0.0), (1.0, 1.0, 1.0))], [(100, 1, 1, (0.0, 0.0, 0.0), (1.0, 0.0, 0.0))]]
    S, heads = 910, 2
    t = random_tensors(S, heads, 120)
    q, k, v = (bf16_to_torch(x).view(S, heads * 128) for x in (t.q, t.k, t.v))
    gq, gk = torch.from_numpy(t.gain_q).cuda(), torch.from_numpy(t.gain_k).cuda()
    with H.Plan(docs, heads) as plan:
        H.h3attn_plan_set_sparse(plan.handle, 256, 3)
        nq = H.h3attn_plan_sparse_info(plan.handle)["n_q_blocks"]
        idx = torch.empty(heads, nq, 3, dtype=torch.int32, device="cuda")
        cnt = torch.empty(heads, nq, dtype=torch.int32, device="cuda")
        qh, kh = torch.empty_like(q), torch.empty_like(k)
        o, lse = W.outputs(S, heads)
        H.h3attn_qk_prologue(plan.handle, q, k, qh, kh, gq, gk)
        H.h3attn_block_select(plan.handle, qh, kh, 3, idx, cnt)
        H.h3attn_forward_sparse(plan.handle, qh, kh, v, idx, cnt, W.flat(o), W.SCALE, lse)
        H.h3attn_get_device_error(plan.handle)
    cu = np.array([0, 810, 910])
    qh, kh, v = (x.view(S, heads, 128) for x in (qh, kh, v))
    want = walks.select(W.f64(qh), W.f64(kh), cu, 256, 3, True)
    assert np.array_equal(idx.cpu().numpy(), want[0]) and np.array_equal(cnt.cpu().numpy(), want[1])
    W.check(o, lse, qh, [kh], walks.sparse_attention(W.f64(qh), W.f64(kh), W.f64(v), cu, 256, *want, W.SCALE))


def test_refusals(lib):
    E = H.H3ATTN_EINVAL
    q, k, v = (W.rows(300, 2, i) for i in range(3))
    with H.Plan(docs_1d([300]), 2) as plan:
        p = plan.handle
        one = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
        assert status(lambda: H.h3attn_plan_sparse_info(p)) == E
        assert status(lambda: H.h3attn_block_select(p, 16, 16, 1, 16, 16, qkv_row_stride=256, stream=0)) == E
        assert status(lambda: H.h3attn_forward_sparse(p, 16, 16, 16, 16, 16, 16, 0.1, qkv_row_stride=256,
                                                      o_row_stride=256, stream=0)) == E
        for bad in ((128, 4), (384, 4), (256, 0), (256, -1), (256, (1 << 20) + 1)):
            assert status(lambda: H.h3attn_plan_set_sparse(p, *bad)) == E
        H.h3attn_plan_set_sparse(p, 256, 4)
        assert status(lambda: H.h3attn_plan_set_sparse(p, 256, 4)) == E  # once per plan
        idx, cnt = one, torch.zeros(2, 2, dtype=torch.int32, device="cuda")
        f = [W.flat(t) for t in (q, k, v)]
        o = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(2, 300, device="cuda")
        for keep in (0, -1, 5):
            assert status(lambda: H.h3attn_block_select(p, f[0], f[1], keep, idx, cnt)) == E
        sel = lambda **kw: H.h3attn_block_select(**{**dict(plan=p, q_hat=f[0].data_ptr(), k_hat=f[1].data_ptr(), keep=2,  # noqa: E731
                                                         block_idx=idx.data_ptr(), block_cnt=cnt.data_ptr(),
                                                         qkv_row_stride=256), **kw})
        fwd = lambda **kw: H.h3attn_forward_sparse(**{**dict(plan=p, q=f[0].data_ptr(), k=f[1].data_ptr(), v=f[2].data_ptr(),  # noqa: E731
                                                           block_idx=idx.data_ptr(), block_cnt=cnt.data_ptr(), o=o.data_ptr(),
                                                           softmax_scale=0.1, lse=lse.data_ptr(), qkv_row_stride=256,
                                                           o_row_stride=256), **kw})
        sel(), fwd()
        for kw in (dict(q_hat=None), dict(k_hat=f[1].data_ptr() + 2), dict(qkv_row_stride=248), dict(qkv_row_stride=260),
                   dict(block_idx=None), dict(block_cnt=cnt.data_ptr() + 2), dict(block_cnt=idx.data_ptr()),
                   dict(block_idx=f[0].data_ptr()), dict(block_cnt=f[1].data_ptr() + 64)):
            assert status(lambda: sel(**kw)) == E, kw
        for kw in (dict(q=None), dict(v=f[2].data_ptr() + 8), dict(block_idx=None), dict(block_idx=idx.data_ptr() + 1),
                   dict(o=f[0].data_ptr()), dict(o=idx.data_ptr()), dict(lse=cnt.data_ptr()), dict(lse=f[2].data_ptr()),
                   dict(softmax_scale=0.0), dict(softmax_scale=float("nan")), dict(o_row_stride=252),
                   dict(qkv_row_stride=128)):
            assert status(lambda: fwd(**kw)) == E, kw
        # tensors of another type, size or layout than the plan's lists
        for bad in (idx.long(), idx[:, :1], idx.transpose(0, 1)):
            with pytest.raises(ValueError):
                H.h3attn_forward_sparse(p, *f, bad, cnt, o, 0.1)
        with pytest.raises(ValueError):
            H.h3attn_block_select(p, f[0], f[1], 2, idx, cnt[:1])
        # tensors that are too short, or not on the device
        for bad in (dict(q=f[0][:299]), dict(o=o[:299]), dict(v=f[2].cpu()), dict(block_idx=idx.cpu())):
            with pytest.raises(ValueError):
                H.h3attn_forward_sparse(**{**dict(plan=p, q=f[0], k=f[1], v=f[2], block_idx=idx, block_cnt=cnt, o=o,
                                                  softmax_scale=0.1), **bad})
        torch.cuda.synchronize()

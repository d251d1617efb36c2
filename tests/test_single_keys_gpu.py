"""That every key a row may see counts exactly once in the sparse and prefix
forwards, at sizes where one key of thousands hides in a tolerance on random
inputs.

Counting: with q = 0 every weight is 2^0, which bf16 holds; with values of +-1
the sums of all keys are whole numbers that fp32 holds.  So o = sum / n, off by
the division and its rounding to bf16 alone (2^-8 and a little of the value: 0
has to be 0), and a key lost, doubled or taken for another moves the sum of some
dim by one, or two: seen wherever the sum is small.  lse = ln n, off by fp32
roundings (2^-20 of it), where a lost key moves it by 1 / n.

Finding: keys are vectors of +-1, and every query is four times the key it looks
for: its score is 45 (128 * 4 / sqrt(128)), that of any other key a sum of 128
signs, of standard deviation 4.  A row's output is the value of its key, off by
the weights of all others (n e^(4 z - 45) for a largest z of 6: below n 2^-29)
and two roundings to bf16; another key's value is off by its whole size."""
import numpy as np
import pytest
import torch

from oracle import walks
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W

pytestmark = pytest.mark.gpu

PREFIX = [
    ([1], 3, 20423), ([1] * 5, 2, 64), ([1] * 64, 21, 5033), ([1] * 200, 1, 12000), ([2] * 50, 2, 12000),
    ([30, 32, 31, 7, 1] * 5, 3, 5000), ([32] * 9, 8, 300), ([1] * 128, 2, 1200), ([17, 405, 1, 64, 129, 300, 33, 700] * 3, 5, 2430),
    ([2000, 2000], 8, 4096), ([31] * 40, 4, 640), ([300] * 12, 20, 1215), ([513, 1, 1100, 257], 3, 129), ([40] * 30, 2, 1),
    ([5033, 2430, 4096], 2, 12960),
]
SPARSE = [
    ([20423], 2, 512, 160), ([20423], 2, 256, 20), ([4096], 5, 512, 8), ([1400, 2576, 488, 3416, 1], 4, 256, 8),
    ([38912], 1, 512, 300), ([64, 80], 2, 256, 3), ([2177, 300], 3, 512, 7), ([12000], 1, 256, 94),
]


def signs(n, heads, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(0, 2, (n, heads, 128), generator=g, device="cuda") * 2 - 1).to(torch.bfloat16)


def check_counts(o, lse, total, n):
    """o [S, H, 128], lse [H, S] against whole sums and numbers of keys per row [S, H]."""
    ref = torch.where(n[..., None] > 0, total / n.clamp(min=1)[..., None], torch.zeros_like(total))
    off = (o.double() - ref).abs() - (2.0 ** -8 + 2.0 ** -20) * ref.abs()
    assert off.max() <= 0, f"row, head, dim {np.unravel_index(int(off.argmax()), off.shape)}: off by {float(off.max()):.2e}"
    want = n.double().log().T
    assert torch.equal(lse == -np.inf, want == -np.inf)
    off = torch.where(want == -np.inf, 0.0, (lse.double() - want).abs() - 2.0 ** -20 * (want + 1))
    assert off.max() <= 0, f"head, row {np.unravel_index(int(off.argmax()), off.shape)}: lse off by {float(off.max()):.2e}"


def random_lists(s, seed):
    """Lists of different lengths in any order; the first and the last tile are in many, some twice."""
    rng = np.random.default_rng(seed)
    idx = np.full((s.heads, s.nq, s.max_blocks), -1, dtype=np.int32)
    cnt = np.zeros((s.heads, s.nq), dtype=np.int32)
    for i, (_, _, a, b) in enumerate(walks.blocks(s.cu, s.q_block)):
        tiles = -(-(b - a) // 128)
        for h in range(s.heads):
            n = int(rng.integers(1, min(tiles, s.max_blocks) + 1))
            pick = rng.permutation(tiles)[:n]
            if n > 2:
                pick[:3] = rng.permutation([0, tiles - 1, pick[3] if n > 3 else 0])
            idx[h, i, :n], cnt[h, i] = pick, n
    return idx, cnt


@pytest.mark.parametrize("lens,heads,prefix", PREFIX)
def test_prefix_counts_every_key_once(lib, lens, heads, prefix):
    p = W.Prefix(lens, heads, prefix)
    q = torch.zeros(p.S, heads, 128, dtype=torch.bfloat16, device="cuda")
    k, kp = W.rows(p.S, heads, 1), W.rows(prefix, heads, 2)
    v, vp = signs(p.S, heads, 3), signs(prefix, heads, 4)
    o, lse = p.forward(q, k, v, kp, vp)
    W.ok(p.plan)
    doc = torch.arange(len(lens), device="cuda").repeat_interleave(torch.tensor(lens, device="cuda"))
    own = torch.zeros(len(lens), heads, 128, dtype=torch.float64, device="cuda").index_add_(0, doc, v.double())
    n = (prefix + torch.tensor(lens, device="cuda"))[doc]
    check_counts(o, lse, vp.double().sum(0) + own[doc], n[:, None].expand(-1, heads))


@pytest.mark.parametrize("lens,heads,q_block,max_blocks", SPARSE)
def test_sparse_counts_every_listed_key_once(lib, lens, heads, q_block, max_blocks):
    s = W.Sparse(lens, heads, q_block, max_blocks)
    q = torch.zeros(s.S, heads, 128, dtype=torch.bfloat16, device="cuda")
    k, v = W.rows(s.S, heads, 1), signs(s.S, heads, 3)
    idx, cnt = random_lists(s, 5)
    s.lists(idx, cnt)
    o, lse = s.forward(q, k, v)
    W.ok(s.plan)
    total = torch.zeros(s.S, heads, 128, dtype=torch.float64, device="cuda")
    n = torch.zeros(s.S, heads, dtype=torch.int64, device="cuda")
    sums = {a: torch.stack([x.double().sum(0) for x in v[a:b].split(128)]) for a, b in zip(s.cu[:-1], s.cu[1:])}
    for i, (q0, q1, a, b) in enumerate(walks.blocks(s.cu, q_block)):
        for h in range(heads):
            pick = torch.from_numpy(idx[h, i, :cnt[h, i]].astype(np.int64)).cuda()
            total[q0:q1, h] = sums[a][pick, h].sum(0)
            n[q0:q1, h] = (b - a - 128 * pick).clamp(max=128).sum()
    check_counts(o, lse, total, n)


def check_found(o, want, n):
    off = (o.double() - want).abs() - (2.0 ** -7 + n * 2.0 ** -29) * (want.abs() + 1)
    assert off.max() <= 0, f"row, head, dim {np.unravel_index(int(off.argmax()), off.shape)}: off by {float(off.max()):.2e}"


@pytest.mark.parametrize("lens,heads,prefix", PREFIX)
def test_prefix_rows_find_their_keys(lib, lens, heads, prefix):
    p = W.Prefix(lens, heads, prefix)
    k, kp, v, vp = signs(p.S, heads, 6), signs(prefix, heads, 7), W.rows(p.S, heads, 8), W.rows(prefix, heads, 9)
    begin = torch.from_numpy(np.repeat(p.cu[:-1], lens)).cuda()[:, None]
    length = torch.from_numpy(np.repeat(lens, lens)).cuda()[:, None]
    head = torch.arange(heads, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(10)
    # the target as a fraction of "the prefix, then the document"; ends and borders for a part of the rows
    at = (torch.rand(p.S, heads, generator=g, device="cuda", dtype=torch.float64) * (prefix + length)).long()
    edge = torch.randint(0, 12, (p.S, heads), generator=g, device="cuda")
    for e, x in enumerate((0, prefix - 1, prefix, prefix + length - 1, min(63, prefix - 1), min(64, prefix - 1))):
        at = torch.where(edge == e, x, at)
    all_k, all_v = torch.cat([kp, k]), torch.cat([vp, v])
    row = torch.where(at < prefix, at, begin + at)  # of [prefix | batch]: document row r lies at prefix + r
    o, _ = p.forward((all_k[row, head].float() * 4).to(torch.bfloat16), k, v, kp, vp)
    W.ok(p.plan)
    check_found(o, all_v[row, head].double(), prefix + max(lens))


@pytest.mark.parametrize("lens,heads,q_block,max_blocks", SPARSE)
def test_sparse_rows_find_their_keys(lib, lens, heads, q_block, max_blocks):
    s = W.Sparse(lens, heads, q_block, max_blocks)
    k, v = signs(s.S, heads, 6), W.rows(s.S, heads, 8)
    idx, cnt = random_lists(s, 11)
    s.lists(idx, cnt)
    row = torch.zeros(s.S, heads, dtype=torch.int64, device="cuda")
    rng = np.random.default_rng(12)
    for i, (q0, q1, a, b) in enumerate(walks.blocks(s.cu, q_block)):
        for h in range(heads):
            tile = rng.choice(idx[h, i, :cnt[h, i]], q1 - q0).astype(np.int64)
            n = np.minimum(128, b - a - 128 * tile)
            key = np.where(rng.random(q1 - q0) < 0.3, rng.choice([0, 1], q1 - q0) * (n - 1), (rng.random(q1 - q0) * n).astype(np.int64))
            row[q0:q1, h] = torch.from_numpy(a + 128 * tile + key).cuda()
    head = torch.arange(heads, device="cuda")
    o, _ = s.forward((k[row, head].float() * 4).to(torch.bfloat16), k, v)
    W.ok(s.plan)
    check_found(o, v[row, head].double(), 128 * max_blocks)


@pytest.mark.parametrize("lens,heads,prefix,few", [
    ([1], 21, 20423, True), ([1] * 64, 21, 5033, True), ([1] * 33, 2, 2200, True), ([32, 31, 1], 2, 300, True),
    ([1, 20], 1, 2200, True), ([1] * 128, 2, 1200, True), ([40] * 30, 2, 300, False), ([33], 2, 300, False),
    ([700, 3, 3, 600], 2, 2430, False)])
def test_which_kernel_a_batch_takes(lib, lens, heads, prefix, few):
    # the few-rows kernel: as many "pairs" as segments, each of at most 32 rows
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    cu = np.concatenate([[0], np.cumsum(lens)])
    units, off, _, _, _ = H.h3attn_walk_list_host(1, cu, heads, prefix, 0, pairs)
    segment_each = len(off) - 1 == len(units) and np.all(units[:, 1] - units[:, 0] <= 32) and np.all(units[:, 7] >= 0)
    assert segment_each == few

"""Rotary blocks of every shape against the fp64 oracle: several rows to a lane group,
more rows than its lane groups hold at once, and as many tokens as a block takes."""
import pytest
import torch

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.test_rotary_gpu import caches, check, positions

pytestmark = pytest.mark.gpu

# rows of a lane group: (tokens of a block) * (heads + key heads [+ key heads]) / 32
SHAPES = [(5033, 21, 21),   # two or three tokens of 42 or 63 rows a block
          (20000, 3, 1),    # sixteen tokens a block, the last one of fewer
          (3, 128, 8),      # a token in two turns
          (2, 300, 20),     # in three
          (700, 65, 33)]    # rows that fill neither their groups nor a turn


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dims", [64, 128])
@pytest.mark.parametrize("n,heads,kv", SHAPES)
def test_rows_of_their_own_and_in_place(lib, n, heads, kv, dims, interleaved):
    q, k, pos = W.rows(n, heads, 1), W.rows(n, kv, 2), positions(n, 1, 3)
    rope = H.h3attn_rope_init(dims, 1e4, interleaved=interleaved)
    f, _ = serving.frequencies(dims, 1e4)
    q2, k2 = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    H.h3attn_rotary(rope, pos.cuda(), q, q2, k, k2)
    check(q2, q, serving.rotate(W.f64(q), pos.numpy(), f, interleaved=interleaved))
    check(k2, k, serving.rotate(W.f64(k), pos.numpy(), f, interleaved=interleaved))
    assert torch.equal(q2[..., dims:], q[..., dims:]) and torch.equal(k2[..., dims:], k[..., dims:])
    H.h3attn_rotary(rope, pos.cuda(), q, q, k, k)
    assert torch.equal(q, q2) and torch.equal(k, k2)


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,kv", SHAPES)
def test_store_with_padding(lib, n, heads, kv, interleaved, head_major):
    page = 16
    pages = -(-n // page) + 2
    kc, vc = caches(pages, page, kv, head_major)
    total, pos = pages * page, positions(n, 1, 14)
    q, k, v = (W.rows(n, h, 11 + i) for i, h in enumerate((heads, kv, kv)))
    slots = torch.randperm(total, generator=torch.Generator().manual_seed(15))[:n].to(torch.int32)
    slots[n // 3::5] = -1
    slots[n // 2::7] = total
    rope = H.h3attn_rope_init(96, 1e5, interleaved=interleaved)
    f, _ = serving.frequencies(96, 1e5)
    want = [kc.clone().reshape(total, kv, 128), vc.clone().reshape(total, kv, 128)]
    there = (slots >= 0) & (slots < total)
    at, rows = slots[there].long().cuda(), there.cuda()
    q2, q3, k2 = torch.full_like(q, float("nan")), q.clone(), torch.empty_like(k)
    H.h3attn_rotary_store(rope, pos.cuda(), q, q2, k, v, H.Cache(kc, vc), slots.cuda())
    check(q2, q, serving.rotate(W.f64(q), pos.numpy(), f, interleaved=interleaved))
    got = kc.reshape(total, kv, 128)
    check(got[at], k[rows], serving.rotate(W.f64(k[rows]), pos.numpy()[:, there.numpy()], f, interleaved=interleaved))
    H.h3attn_rotary(rope, pos.cuda(), None, None, k, k2)
    want[0][at], want[1][at] = k2[rows], v[rows]
    assert torch.equal(got, want[0]) and torch.equal(vc.reshape(total, kv, 128), want[1])
    # q in place, the same rows again
    H.h3attn_rotary_store(rope, pos.cuda(), q3, q3, k, v, H.Cache(kc, vc), slots.cuda())
    assert torch.equal(q3, q2) and torch.equal(kc.reshape(total, kv, 128), want[0]) and torch.equal(vc.reshape(total, kv, 128), want[1])

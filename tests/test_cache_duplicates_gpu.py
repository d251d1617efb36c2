"""Moves that name a destination several times: of a group's pairs that do, the last
one's row stays, whole, in k and in v and in every head."""
import numpy as np
import pytest
import torch

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.test_rotary_gpu import caches

pytestmark = pytest.mark.gpu


def moved(kc, vc, src, dst):
    pages, page, kv = kc.shape[:3]
    flat = [W.f64(c.float()).reshape(pages * page, kv, 128) for c in (kc, vc)]
    want = [serving.moved(x, src, dst) for x in flat]
    H.h3attn_cache_move(H.Cache(kc, vc), torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    for c, w in zip((kc, vc), want):
        assert np.array_equal(W.f64(c.float()).reshape(w.shape), w)


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("groups,width,page,kv,targets", [(3, 2, 8, 1, 1), (40, 16, 16, 2, 3), (20, 17, 8, 3, 5), (30, 64, 64, 8, 2), (9, 65, 16, 2, 40),
                                                          (50, 256, 7, 4, 1), (10, 256, 32, 2, 100)])
def test_the_last_of_equal_destinations_stays(lib, groups, width, page, kv, targets, head_major):
    kc, vc = caches(-(-2 * groups * width // page) + 1, page, kv, head_major)
    total, g = kc.shape[0] * page, np.random.default_rng(3)
    for _ in range(5):
        own = g.permutation(total)[:2 * groups * width].reshape(groups, 2 * width)  # slots of one group only
        src = np.stack([g.choice(x, width) for x in own]).astype(np.int32)
        dst = np.stack([g.choice(x[:targets], width) for x in own]).astype(np.int32)
        moved(kc, vc, src, dst)


@pytest.mark.parametrize("width", [3, 33, 256])
def test_pairs_that_are_left_out_do_not_count(lib, width):
    # behind the last pair that is one, others name its destination without a source, or a source without a destination
    kc, vc = caches(2 * width, 8, 2, False)
    total = kc.shape[0] * 8
    src = np.arange(width, dtype=np.int32)[None] + width
    dst = np.zeros((1, width), dtype=np.int32)
    keep = width // 2
    src[0, keep + 1:] = [(-1, total, 2 ** 31 - 1, -2 ** 31)[i % 4] for i in range(width - keep - 1)]
    moved(kc, vc, src, dst)
    moved(kc, vc, np.where(src < 0, 5, src).astype(np.int32), np.where(np.arange(width) > keep, -1, dst).astype(np.int32))

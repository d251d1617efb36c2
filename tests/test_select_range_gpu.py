"""Block selection over the range of its inputs' magnitudes, against the fp64
oracle: ties and near ties that an fp32 sum cannot tell, from subnormal key
means on to products beyond fp32's range.

What is kept is a discrete answer, so everything is compared for equality.  The
scores of a tie are sums of the same 128 products in another order; with q all
ones the products are fp32 numbers whose exponents differ by less than 2^20, so
their sums are exact in fp64 in any order, and the lower tile is the answer."""
import numpy as np
import pytest
import torch

from oracle import walks
from tests import walk_cases as W

pytestmark = pytest.mark.gpu

HEADS = 64


@pytest.mark.parametrize("tiles", [2, 40])  # 40: more tied tiles than a warp ranks at once
@pytest.mark.parametrize("log2", [0, -60, -78, -85, -100, -120, 60, 100])
def test_permuted_key_means_tie(lib, tiles, log2):
    s = W.Sparse([128 * tiles], HEADS, 512, tiles)
    first = (W.rows(128, HEADS, 1).float() * 2.0 ** log2).to(torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(2)
    k = torch.cat([first] + [first[:, :, torch.randperm(128, generator=gen, device="cuda")] for _ in range(tiles - 1)])
    q = torch.ones_like(k)
    for keep in (1, tiles - 1):
        idx, cnt = s.select(q, k, keep)
        assert np.all(cnt == keep)
        assert np.array_equal(idx[:, :, :keep], np.broadcast_to(np.arange(keep), idx[:, :, :keep].shape))


@pytest.mark.parametrize("log2_q,log2_k", [(0, -80), (0, -100), (-50, -50), (0, 90), (60, 60), (100, 100)])
def test_scores_whose_large_terms_cancel(lib, log2_q, log2_k):
    # M + what they share + small - M, the small terms 2^-26 of M
    k = W.rows(128, 1, 5).repeat(8, 1, 1)
    k[:, :, 0], k[:, :, 4] = 2.0 ** 11, -(2.0 ** 11)
    for t in range(8):
        k[128 * t:128 * t + 128, 0, 2] = 2.0 ** -12 * ((5 * t) % 8)
    q = W.rows(1024, 1, 6)
    q[:, :, 0], q[:, :, 2], q[:, :, 4] = 1.0, 1.0, 1.0
    q, k = ((x.float() * 2.0 ** e).to(torch.bfloat16) for x, e in ((q, log2_q), (k, log2_k)))
    s = W.Sparse([1024], 1, 512, 3)
    idx, cnt = s.select(q, k, 3)
    want = walks.select(W.f64(q), W.f64(k), s.cu, 512, 3, False)
    assert np.array_equal(idx, want[0]) and np.array_equal(cnt, want[1])
    assert idx[0, 0].tolist() == [1, 3, 6]  # (5 t) % 8 = 5, 7, 6: the largest three


@pytest.mark.parametrize("log2_q,log2_k", [(0, -110), (-60, -60), (-126, 0), (-70, 0), (112, -20), (112, 112)])
@pytest.mark.parametrize("lens", [[1500, 129], [300 * 128 - 5]])
def test_random_inputs_of_any_magnitude(lib, lens, log2_q, log2_k):
    s = W.Sparse(lens, 2, 256, 9)
    # (|rows| below 8: the largest element stays below the documented 2^112 where the scale is 2^-3 of it)
    q, k = ((W.rows(s.S, 2, 20 + i).float() * 2.0 ** (e - 3)).to(torch.bfloat16) for i, e in enumerate((log2_q, log2_k)))
    for own in (False, True):
        idx, cnt = s.select(q, k, 9, keep_own=own)
        want = walks.select(W.f64(q), W.f64(k), s.cu, 256, 9, own)
        assert np.array_equal(idx, want[0]) and np.array_equal(cnt, want[1])

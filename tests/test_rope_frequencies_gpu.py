"""Frequencies of a program's own in place of those that h3attn_rope_init found: a ramp
over pair indices, and a table."""
import math

import numpy as np
import pytest

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.test_rotary_gpu import check, positions


def index_ramp(dims, base, factor, original_len, fast=32.0, slow=1.0):
    """f (g + (1 - g)/factor), g falling from 1 to 0 over the pair's index between those that turn `fast` and `slow` times."""
    at = [dims * math.log(original_len / (2 * math.pi * b)) / (2 * math.log(base)) for b in (fast, slow)]
    low, high = max(0, math.floor(at[0])), min(dims - 1, math.ceil(at[1]))
    j = np.arange(dims // 2)
    g = 1 - np.clip((j - low) / (high - low), 0, 1)
    return float(base) ** (-2.0 * j / dims) * (g + (1 - g) / factor)


def given(f, amplitude, interleaved=False):
    rope = H.h3attn_rope_init(2 * len(f), 1e4, interleaved=interleaved, amplitude=amplitude)
    for j, x in enumerate(f):
        rope.turns[j] = int(x / (2 * math.pi) * 2 ** 64)
    return rope


def test_the_two_ramps_differ(lib):
    # (what the documentation says: by parts ramps over turns)
    f, _ = serving.frequencies(128, 1e6, "parts", 4.0, 32768)
    rope, own = H.h3attn_rope_init(128, 1e6, scaling="parts", factor=4.0, original_len=32768), index_ramp(128, 1e6, 4.0, 32768)
    got = np.array([rope.turns[j] / 2.0 ** 64 * 2 * math.pi for j in range(64)])
    assert np.allclose(got, f, rtol=1e-12, atol=0)
    assert abs(f[32] - 3.5e-4) < 5e-6 and abs(own[32] - 6.0e-4) < 5e-6


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("f,amplitude", [(index_ramp(128, 1e6, 4.0, 32768), 0.1 * math.log(4.0) + 1), (index_ramp(64, 1e4, 8.0, 4096), 1.0),
                                         (np.geomspace(3.0, 1e-7, 24), 0.5), (np.zeros(8), 2.0)])
def test_frequencies_of_ones_own(lib, f, amplitude, interleaved):
    n, dims = 300, 2 * len(f)
    q, k, pos = W.rows(n, 6, 1), W.rows(n, 2, 2), positions(n, 1, 3, far=100000)
    q2, k2 = q.clone(), k.clone()
    H.h3attn_rotary(given(f, amplitude, interleaved), pos.cuda(), q, q2, k, k2)
    for got, x in ((q2, q), (k2, k)):
        check(got, x, serving.rotate(W.f64(x), pos.numpy(), f, amplitude, interleaved=interleaved), amplitude)

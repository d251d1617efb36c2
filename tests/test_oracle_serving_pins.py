"""Pins of the oracle of rotary positions, causal and tree attention and cache
moves: closed forms and brute force that share nothing with it."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention, serving


def test_unit_vectors_turn_as_the_closed_form():
    f, amplitude = serving.frequencies(64, 10000.0)
    assert amplitude == 1.0 and f[0] == 1.0 and math.isclose(f[16], 10000.0 ** -0.5, rel_tol=1e-15)
    for inter, lo, hi in ((False, 5, 37), (True, 10, 11)):
        x = np.zeros((1, 1, 128))
        x[0, 0, lo] = 1.0
        y = serving.rotate(x, [[3]], f, interleaved=inter)[0, 0]
        assert math.isclose(y[lo], math.cos(3 * f[5])) and math.isclose(y[hi], math.sin(3 * f[5]))
        assert np.count_nonzero(y) == 2
        z = serving.rotate(x, [[3]], f, interleaved=inter, inverse=True)[0, 0]
        assert math.isclose(z[hi], -y[hi])


def test_scores_depend_on_distance_and_other_dims_pass():
    rng = np.random.default_rng(0)
    f, _ = serving.frequencies(96, 1e6)
    q, k = rng.standard_normal((2, 1, 1, 128))
    dot = lambda p, r: float((serving.rotate(q, [[p]], f) * serving.rotate(k, [[r]], f)).sum())  # noqa: E731
    assert math.isclose(dot(7, 3), dot(1004, 1000), rel_tol=1e-9)
    assert np.array_equal(serving.rotate(q, [[9]], f)[..., 96:], q[..., 96:])


def test_axes_take_their_own_positions():
    f, _ = serving.frequencies(32, 100.0)
    x = np.random.default_rng(1).standard_normal((1, 1, 128))
    axes = [j % 3 for j in range(16)]
    y = serving.rotate(x, [[4], [0], [0]], f, axes=axes)
    same = [j for j in range(16) if axes[j] != 0]
    assert np.array_equal(y[0, 0, same], x[0, 0, same])
    assert not np.isclose(y[0, 0, 3], x[0, 0, 3])


def test_scalings():
    f, _ = serving.frequencies(128, 1e4)
    assert np.allclose(serving.frequencies(128, 1e4, "linear", 4.0)[0], f / 4)
    n, _ = serving.frequencies(128, 1e4, "ntk", 4.0)
    assert math.isclose(n[0], 1.0) and math.isclose(n[63], f[63] / 4, rel_tol=1e-12)  # the lowest as linear
    p, a = serving.frequencies(128, 1e4, "parts", 4.0, original_len=4096)
    turns = 4096 * f / (2 * np.pi)
    assert np.array_equal(p[turns > 32], f[turns > 32]) and np.allclose(p[turns < 1], f[turns < 1] / 4)
    assert np.all(np.diff(p) < 0) and math.isclose(a, 0.1 * math.log(4) + 1)


def test_causal_against_the_packed_oracle_and_brute_force():
    rng = np.random.default_rng(2)
    cu = np.array([0, 1, 6, 15])
    q, k, v = rng.standard_normal((15, 4, 8)), rng.standard_normal((15, 2, 8)), rng.standard_normal((15, 2, 8))
    o, wv, lse = serving.causal_attention(q, k, v, cu, 0.3)
    full, full_lse = attention.attention(q, k.repeat(2, 1), v.repeat(2, 1), cu, 0.3)
    for last in cu[1:] - 1:  # the last row of a document sees all of it
        assert np.allclose(o[last], full[last], atol=1e-13) and np.allclose(lse[:, last], full_lse[:, last], atol=1e-13)
    for i, a in ((0, 0), (3, 1), (9, 6)):
        for h in range(4):
            w = [math.exp(0.3 * sum(q[i, h] * k[j, h // 2])) for j in range(a, i + 1)]
            want = sum(x * v[j, h // 2] for x, j in zip(w, range(a, i + 1))) / sum(w)
            assert np.allclose(o[i, h], want, atol=1e-13) and math.isclose(lse[h, i], math.log(sum(w)), abs_tol=1e-13)
    assert np.all(wv >= np.abs(o) - 1e-15)
    some, _, _ = serving.causal_attention(q, k, v, cu, 0.3, rows=[4, 14])
    assert np.allclose(some, o[[4, 14]], atol=1e-13)  # (other shapes, another order of summation)


def test_a_chain_is_causal_and_an_empty_mask_is_zero():
    rng = np.random.default_rng(3)
    page, n, T = 4, 7, 5
    table = np.array([[3, 0, 2]])
    kc, vc = rng.standard_normal((2, 4, page, 1, 8))
    at = serving.slots_of(table[0], n + T, page)
    assert at.tolist() == [12, 13, 14, 15, 0, 1, 2, 3, 8, 9, 10, 11]
    q = rng.standard_normal((T, 2, 8))
    o, _, lse = serving.tree_attention(q, kc, vc, table, [n], [0, T], None, 0.5)
    whole = np.concatenate([rng.standard_normal((n, 2, 8)), q])
    ref, _, ref_lse = serving.causal_attention(whole, kc.reshape(-1, 1, 8)[at], vc.reshape(-1, 1, 8)[at], [0, n + T], 0.5)
    assert np.allclose(o, ref[n:]) and np.allclose(lse, ref_lse[:, n:])
    o, wv, lse = serving.tree_attention(q, kc, vc, table, [0], [0, T], [0, 1, 3, 8, 0], 0.5)
    assert not o[[0, 4]].any() and not wv[0].any() and np.isneginf(lse[:, [0, 4]]).all()
    assert np.allclose(o[3], vc.reshape(-1, 8)[at[3]])


def test_moves_read_before_they_write():
    rows = np.arange(10)
    assert serving.moved(rows, [[5, 0, -1, 3]], [[0, 5, 2, 11]]).tolist() == [5, 1, 2, 3, 4, 0, 6, 7, 8, 9]
    assert serving.moved(rows, [[1, 2], [7, 8]], [[2, 3], [8, 9]]).tolist() == [0, 1, 1, 2, 4, 5, 6, 7, 7, 8]


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
@pytest.mark.parametrize("dims", [16, 96, 128])
def test_the_library_keeps_the_same_frequencies(lib, dims, scaling):
    f, a = serving.frequencies(dims, 5e5, scaling, 8.0, original_len=8192)
    r = lib.h3attn_rope_init(dims, 5e5, scaling=scaling, factor=8.0, original_len=8192)
    for j in range(dims // 2):
        # (a few roundings of fp64 on either side, and the cut to 2^-64)
        got = Fraction(int(r.turns[j]), 2 ** 64)
        want = Fraction(float(f[j])) / Fraction(2 * math.pi)
        assert abs(got - want) <= want * Fraction(16, 2 ** 53) + Fraction(1, 2 ** 64)
    assert math.isclose(r.amplitude, a, rel_tol=2 ** -24)

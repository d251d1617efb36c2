"""Oracle: rotary positions, causal attention with grouped heads, attention for
trees of drafts over a paged cache, and row moves within one; fp64 (rows as
fp64 arrays), from the definitions in ``include/h3attn.h``.

    rotary:  pair (a, b) -> A (a cos t - b sin t, b cos t + a sin t), t = p f_j;
    causal:  row i of a document attends to the document's rows up to i, query
             head h to key head h // group;
    tree:    a draft attends to its sequence's context and to the drafts of its
             mask, all looked up through the sequence's pages; o = 0 and lse =
             -inf where there is nothing;
    moves:   new[dst] = old[src], group by group.

Each attention also returns sum_j w_j |v_j| (w the softmax weights), the scale of
the error that rounding the weights to bf16 may cause.

Parity: pinned (angles against exact rational arithmetic on short positions and
closed forms; causal attention against the packed oracle's last row and a brute
force; a tree that is a chain against causal attention).
"""
from __future__ import annotations

import numpy as np


def frequencies(dims, base, scaling="none", factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """f_j of the dims/2 pairs, and the default amplitude."""
    j = np.arange(dims // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (dims / (dims - 2))
    f = base ** (-2.0 * j / dims)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        turns = original_len * f / (2 * np.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return f * (g + (1 - g) / factor), 0.1 * np.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, f, amplitude=1.0, axes=None, interleaved=False, inverse=False):
    """x fp64 [n, heads, 128], pos [n_axes, n] whole numbers."""
    d = 2 * len(f)
    axes = np.zeros(len(f), dtype=np.int64) if axes is None else np.asarray(axes)
    t = np.asarray(pos, dtype=np.float64)[axes].T * f                 # [n, d/2]
    c, s = amplitude * np.cos(t)[:, None], amplitude * np.sin(t)[:, None]
    if inverse:
        s = -s
    lo = np.arange(0, d, 2) if interleaved else np.arange(d // 2)
    hi = lo + 1 if interleaved else lo + d // 2
    y = np.array(x, dtype=np.float64)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def _attend(q, k, v, seen, scale):
    """Rows q [n, D] over keys k [m, D], the pairs of `seen` [n, m]: o, sum w|v|, lse."""
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, keepdims=True, initial=-np.inf)
    m0 = np.where(np.isneginf(m), 0.0, m)
    e = np.where(seen, np.exp(np.where(seen, s, 0.0) - m0), 0.0)
    total = e.sum(axis=1, keepdims=True)
    w = e / np.where(total > 0, total, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(total))[:, 0]
    return w @ v, w @ np.abs(v), lse


def causal_attention(q, k, v, cu, scale, rows=None):
    """(o, sum w|v|, lse) of all rows, or of the given ones: q [S, H, D], k and v [S, Hkv, D]."""
    S, H, D = q.shape
    group = H // k.shape[1]
    rows = np.arange(S) if rows is None else np.asarray(rows)
    o, wv, lse = np.zeros((len(rows), H, D)), np.zeros((len(rows), H, D)), np.zeros((H, len(rows)))
    for a, b in zip(cu[:-1], cu[1:]):
        at = np.nonzero((rows >= a) & (rows < b))[0]
        if at.size == 0:
            continue
        i = rows[at]
        seen = np.arange(a, b) <= i[:, None]
        for h in range(H):
            o[at, h], wv[at, h], lse[h, at] = _attend(q[i, h], k[a:b, h // group], v[a:b, h // group], seen, scale)
    return o, wv, lse


def slots_of(table, n, page):
    """Slots of a sequence's first n rows."""
    i = np.arange(n)
    return np.asarray(table, dtype=np.int64)[i // page] * page + i % page


def tree_attention(q, k_cache, v_cache, table, ctx, cu, masks, scale):
    """(o, sum w|v|, lse): caches [pages, page, Hkv, D], masks a list of whole numbers or None."""
    S, H, D = q.shape
    page, kv = k_cache.shape[1:3]
    o, wv, lse = np.zeros((S, H, D)), np.zeros((S, H, D)), np.zeros((H, S))
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        n, T = int(ctx[b]), int(e - a)
        at = slots_of(table[b], n + T, page)
        k, v = (c.reshape(-1, kv, D)[at] for c in (k_cache, v_cache))
        seen = np.ones((T, n + T), dtype=bool)
        for i in range(T):
            word = (1 << (i + 1)) - 1 if masks is None else int(masks[a + i])
            seen[i, n:] = [word >> j & 1 for j in range(T)]
        for h in range(H):
            g = h // (H // kv)
            o[a:e, h], wv[a:e, h], lse[h, a:e] = _attend(q[a:e, h], k[:, g], v[:, g], seen, scale)
    return o, wv, lse


def moved(rows, src, dst):
    """rows [slots, ...] after the moves of every group."""
    new = rows.copy()
    for s, d in zip(src, dst):
        for x, y in zip(s, d):
            if 0 <= x < len(rows) and 0 <= y < len(rows):
                new[y] = rows[x]
    return new

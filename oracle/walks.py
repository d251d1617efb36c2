"""Oracle: block selection, block-sparse attention and attention with a shared
prefix, fp64, from the definitions in ``include/h3attn.h``.

Blocks: document [a, b) has query blocks of q_block rows and key tiles of 128
rows, both counted from a; query blocks are numbered over all documents.

    score_ij = <mean of block i's q rows, mean of tile j's k rows>
               (means rounded once to fp32), the `keep` largest kept, ties to
               the lower tile, tiles overlapping the block first if keep_own;
    sparse:  softmax attention of a row over the keys of the tiles listed for
             its block (a tile listed twice counts twice); o = 0 and lse = -inf
             where nothing is listed;
    prefix:  softmax attention of a row over the prefix's rows and its own
             document's.

Each attention also returns sum_j w_j |v_j| (w the softmax weights), the scale
of the error that rounding the weights to bf16 may cause.

Parity: pinned (all tiles listed, or a prefix that is the rest of the document,
reproduce the packed attention; selection against exact rational arithmetic).
"""
from __future__ import annotations

import numpy as np

TILE = 128


def blocks(cu, q_block):
    """(first row, end, document begin, document end) of every query block."""
    return [(r, min(r + q_block, int(b)), int(a), int(b))
            for a, b in zip(cu[:-1], cu[1:]) for r in range(int(a), int(b), q_block)]


def scores(q, k, block):
    """fp64 scores [H, tiles] of one query block: q, k fp64 [S, H, D]."""
    q0, q1, a, b = block
    qm = q[q0:q1].mean(axis=0).astype(np.float32).astype(np.float64)                # [H, D]
    km = np.stack([k[t:min(t + TILE, b)].mean(axis=0) for t in range(a, b, TILE)])  # [T, H, D]
    return np.einsum("hd,thd->ht", qm, km.astype(np.float32).astype(np.float64))


def pick(score, keep, own=None):
    """Ascending indices of the `keep` largest scores (NaN below every number,
    ties to the lower index; the tiles of range `own` first)."""
    def rank(j):
        if own is not None and j in own:
            return (-2, 0.0)
        return (0, 0.0) if np.isnan(score[j]) else (-1, -score[j])
    return sorted(sorted(range(len(score)), key=rank)[:keep])


def select(q, k, cu, q_block, keep, keep_own, width=None):
    """block_idx int32 [H, NQ, width] (width defaults to keep) and block_cnt."""
    bl = blocks(cu, q_block)
    H = q.shape[1]
    idx = np.full((H, len(bl), width or keep), -1, dtype=np.int32)
    cnt = np.zeros((H, len(bl)), dtype=np.int32)
    for i, block in enumerate(bl):
        s = scores(q, k, block)
        q0, q1, a, _ = block
        own = range((q0 - a) // TILE, -(-(q1 - a) // TILE)) if keep_own else None
        for h in range(H):
            best = pick(s[h], keep, own)
            idx[h, i, :len(best)] = best
            cnt[h, i] = len(best)
    return idx, cnt


def _attend(q, keys, vals, scale):
    """o, sum w |v| and lse of rows q over the given keys (two-pass softmax)."""
    if len(keys) == 0:
        z = np.zeros((len(q), vals.shape[1]))
        return z, z.copy(), np.full(len(q), -np.inf)
    s = scale * (q @ keys.T)
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    total = e.sum(axis=1, keepdims=True)
    w = e / total
    return w @ vals, w @ np.abs(vals), (m + np.log(total))[:, 0]


def sparse_attention(q, k, v, cu, q_block, idx, cnt, scale):
    """(o [S, H, D], sum w|v| [S, H, D], lse [H, S]) over the listed tiles."""
    S, H, D = q.shape
    o, wv, lse = np.zeros((S, H, D)), np.zeros((S, H, D)), np.zeros((H, S))
    for i, (q0, q1, a, b) in enumerate(blocks(cu, q_block)):
        for h in range(H):
            keys = [np.arange(a + TILE * t, min(a + TILE * t + TILE, b)) for t in idx[h, i, :max(0, cnt[h, i])]]
            keys = np.concatenate(keys) if keys else np.zeros(0, dtype=np.int64)
            o[q0:q1, h], wv[q0:q1, h], lse[h, q0:q1] = _attend(q[q0:q1, h], k[keys, h], v[keys, h], scale)
    return o, wv, lse


def prefix_attention(q, k, v, k_prefix, v_prefix, cu, scale):
    """(o, sum w|v|, lse) of documents that share a prefix."""
    S, H, D = q.shape
    o, wv, lse = np.zeros((S, H, D)), np.zeros((S, H, D)), np.zeros((H, S))
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(H):
            keys = np.concatenate([k_prefix[:, h], k[a:b, h]])
            vals = np.concatenate([v_prefix[:, h], v[a:b, h]])
            o[a:b, h], wv[a:b, h], lse[h, a:b] = _attend(q[a:b, h], keys, vals, scale)
    return o, wv, lse

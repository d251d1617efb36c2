"""Inputs, runs and tolerances of the block-sparse and shared-prefix tests."""
from __future__ import annotations

import numpy as np
import torch

from packed_varlen_non_gb300 import h3attn as H
from tests.gpu_cases import docs_1d

SCALE = 1.0 / np.sqrt(128.0)


def rows(n, heads, seed, scale=1.0):
    """bf16 rows [n, heads, 128] on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(n, heads, 128, generator=g, device="cuda")).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def strided(t, stride, guard=float("nan")):
    """The same rows in a wider buffer (row stride `stride` elements), `guard` around them."""
    n, h, _ = t.shape
    buf = torch.full((n, stride), guard, dtype=t.dtype, device="cuda")
    buf[:, :h * 128] = t.reshape(n, h * 128)
    return buf[:, :h * 128]


def check(o, lse, q, keys, want, what=""):
    """o [S, H, 128] and lse [H, S] (device) against the oracle's (o, sum w|v|,
    lse).  Per element: the weights are rounded to bf16 before they multiply v
    (half a step, 2^-8 of each w_j |v_j|), the result once more (2^-8 |o|); a
    score is a sum of 128 products in fp32, off by at most 128 * 2^-23 times
    |q| |k| softmax_scale (a step per addition), and moves numerator and
    denominator of a weight by that share each, and so does lse; exponentials
    and the running sums' own roundings are below 2^-20."""
    ref, wv, ref_lse = want
    norm = float(np.linalg.norm(f64(q), axis=-1).max()) * max(
        [float(np.linalg.norm(f64(k), axis=-1).max()) for k in keys if len(k)])
    score = 128 * 2.0 ** -23 * norm * SCALE
    got = f64(o)
    tol = (2.0 ** -8 + 2 * score + 2.0 ** -20) * wv + 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * wv
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs out of tolerance, first at {np.argwhere(bad)[0]}"
    if lse is not None:
        got = f64(lse)
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(got), empty), f"{what}: -inf rows differ"
        err = np.abs(got[~empty] - ref_lse[~empty]) - 2.0 ** -20 * np.abs(ref_lse[~empty])
        assert err.size == 0 or err.max() <= score + 2.0 ** -20, f"{what}: lse off by {err.max():.2e}"


class Sparse:
    """A plan with sparse lists, its list tensors and calls."""

    def __init__(self, lens, heads, q_block, max_blocks):
        self.lens, self.heads, self.q_block, self.max_blocks = lens, heads, q_block, max_blocks
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        self.S = int(self.cu[-1])
        self.plan = H.Plan(docs_1d(lens), heads)
        H.h3attn_plan_set_sparse(self.plan.handle, q_block, max_blocks)
        self.nq = H.h3attn_plan_sparse_info(self.plan.handle)["n_q_blocks"]
        self.idx = torch.full((heads, self.nq, max_blocks), -7, dtype=torch.int32, device="cuda")
        self.cnt = torch.full((heads, self.nq), -7, dtype=torch.int32, device="cuda")

    def select(self, q, k, keep, keep_own=False):
        H.h3attn_block_select(self.plan.handle, flat(q), flat(k), keep, self.idx, self.cnt, keep_own=keep_own)
        return self.idx.cpu().numpy(), self.cnt.cpu().numpy()

    def lists(self, idx, cnt):
        self.idx.copy_(torch.from_numpy(idx))
        self.cnt.copy_(torch.from_numpy(cnt))

    def forward(self, q, k, v, o=None, lse=None, with_lse=True, stream=None):
        o, lse = outputs(self.S, self.heads, o, lse)
        H.h3attn_forward_sparse(self.plan.handle, flat(q), flat(k), flat(v), self.idx, self.cnt, flat(o), SCALE,
                                lse if with_lse else None, stream=stream)
        return o, lse


class Prefix:
    """A plan with a shared prefix."""

    def __init__(self, lens, heads, prefix):
        self.lens, self.heads, self.prefix = lens, heads, prefix
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        self.S = int(self.cu[-1])
        self.plan = H.Plan(docs_1d(lens), heads)
        H.h3attn_plan_set_prefix(self.plan.handle, prefix)

    def forward(self, q, k, v, kp, vp, o=None, lse=None, with_lse=True, stream=None):
        o, lse = outputs(self.S, self.heads, o, lse)
        H.h3attn_forward_prefix(self.plan.handle, flat(q), flat(k), flat(v), flat(kp), flat(vp), flat(o), SCALE,
                                lse if with_lse else None, stream=stream)
        return o, lse


def flat(t):
    """[n, H, 128] -> [n, H * 128] (a strided 2D view stays as it is)."""
    return t if t.dim() == 2 else t.reshape(t.shape[0], -1)


def outputs(S, heads, o=None, lse=None):
    if o is None:
        o = torch.full((S, heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    if lse is None:
        lse = torch.full((heads, S), float("nan"), dtype=torch.float32, device="cuda")
    return o, lse


def ok(plan):
    H.h3attn_get_device_error(plan.handle)

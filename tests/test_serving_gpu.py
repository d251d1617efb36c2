"""The calls of a text tower together, as a program uses them: prompts rotated,
stored into pages and attended causally, then steps of single tokens and of
drafted trees over the cache, their accepted drafts moved up -- against one
causal attention over every finished sequence in fp64."""
import numpy as np
import pytest
import torch

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d

pytestmark = pytest.mark.gpu

PAGE, CAP = 16, 24  # rows and pages of a sequence


@pytest.mark.parametrize("heads,kv,scaling", [(8, 2, "none"), (7, 1, "parts"), (3, 3, "ntk")])
@pytest.mark.parametrize("lens", [[5, 130, 1], [300]])
def test_a_prompt_then_steps_then_trees(lib, heads, kv, scaling, lens):
    n_seq, S = len(lens), sum(lens)
    rope = H.h3attn_rope_init(128, 1e4, scaling=scaling, factor=2.0, original_len=256)
    pages = n_seq * CAP
    kc, vc = (torch.full((pages, PAGE, kv, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = H.Cache(kc, vc)
    table = np.random.default_rng(1).permutation(pages).reshape(n_seq, CAP).astype(np.int32)
    d_table = torch.from_numpy(table).cuda()
    d_ctx = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    known = [[] for _ in lens]   # every sequence's finished rows: (q rotated, k rotated, v, o, lse)

    def project(rows, seed):
        """What a fused projection of the tokens gives: q, k, v in one buffer."""
        buf = W.rows(rows, heads + 2 * kv, seed)
        return buf[:, :heads], buf[:, heads:heads + kv], buf[:, heads + kv:]

    def ints(x):
        return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")

    # the prompts: keys go to the cache, and (rotated again, beside it) to the causal forward
    q, k, v = project(S, 10)
    pos = np.concatenate([np.arange(n) for n in lens])
    slots = np.concatenate([serving.slots_of(table[b], n, PAGE) for b, n in enumerate(lens)])
    q2, k2 = torch.empty(S, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(S, kv, 128, dtype=torch.bfloat16, device="cuda")
    H.h3attn_rotary_store(rope, ints(pos), q, q2, k, v, cache, ints(slots))
    H.h3attn_rotary(rope, ints(pos), None, None, k, k2)
    o, lse = W.outputs(S, heads)
    with H.Plan(docs_1d(lens), heads) as plan:
        H.h3attn_plan_set_causal(plan.handle, kv)
        H.h3attn_forward_causal(plan.handle, q2, k2, v.contiguous(), o, W.SCALE, lse)
        W.ok(plan)
    at = 0
    for b, n in enumerate(lens):
        known[b] += [(q2[i], k2[i], v[i], o[i], lse[:, i]) for i in range(at, at + n)]
        at += n

    # steps: one token a sequence, then trees of 6 of which a path is accepted
    rng = np.random.default_rng(2)
    for step, drafts in enumerate([1, 1, 6, 6, 1]):
        with H.Plan(docs_1d([drafts] * n_seq), heads) as plan:
            H.h3attn_plan_set_tree(plan.handle, kv)
            rows = n_seq * drafts
            parent = [-1] + [int(rng.integers(0, i)) for i in range(1, drafts)]
            mask, depth = [], []
            for i, p in enumerate(parent):
                mask.append((mask[p] if p >= 0 else 0) | 1 << i)
                depth.append(depth[p] + 1 if p >= 0 else 0)
            done = [len(x) for x in known]
            slots = [serving.slots_of(table[b], done[b] + drafts, PAGE)[done[b]:] for b in range(n_seq)]
            q, k, v = project(rows, 100 + step)
            q2, k2 = torch.empty(rows, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, kv, 128, dtype=torch.bfloat16, device="cuda")
            pos = ints(np.concatenate([done[b] + np.array(depth) for b in range(n_seq)]))
            d_ctx.copy_(ints(done))
            H.h3attn_rotary_store(rope, pos, q, q2, k, v, cache, ints(np.concatenate(slots)))
            H.h3attn_rotary(rope, pos, None, None, k, k2)
            o, lse = W.outputs(rows, heads)
            H.h3attn_forward_tree(plan.handle, q2, cache, d_table, d_ctx, o, W.SCALE, lse,
                                  tree_mask=torch.tensor(mask * n_seq, device="cuda"))
            W.ok(plan)
            # the path to the deepest draft is accepted
            node, path = int(np.argmax(depth)), []
            while node >= 0:
                path.insert(0, node)
                node = parent[node]
            src = ints([[slots[b][i] for i in path] for b in range(n_seq)])
            dst = ints([[slots[b][i] for i in range(len(path))] for b in range(n_seq)])
            H.h3attn_cache_move(cache, src, dst)
            for b in range(n_seq):
                known[b] += [(q2[b * drafts + i], k2[b * drafts + i], v[b * drafts + i], o[b * drafts + i], lse[:, b * drafts + i])
                             for i in path]

    # every row that any call computed is that of one causal attention over its finished sequence
    for b in range(n_seq):
        qs, ks, vs, os = (torch.stack([row[i] for row in known[b]]) for i in range(4))
        lses = torch.stack([row[4] for row in known[b]], 1)
        want = serving.causal_attention(*(W.f64(x) for x in (qs, ks, vs)), [0, len(known[b])], W.SCALE)
        W.check(os, lses, qs, [ks], want, f"sequence {b}")
        at = torch.from_numpy(serving.slots_of(table[b], len(known[b]), PAGE)).cuda()
        assert torch.equal(kc.view(-1, kv, 128)[at], ks) and torch.equal(vc.view(-1, kv, 128)[at], vs)


def test_calls_from_several_host_threads_and_on_other_streams(lib):
    # each thread a plan, a cache and a stream of its own; the rotary tables are host data that all share
    import threading
    rope, heads, kv, n = H.h3attn_rope_init(64, 1e4, interleaved=True), 4, 2, 200
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    x = [W.rows(n, h, 40 + i) for i, h in enumerate((heads, kv, kv))]
    ref_q, ref_k = torch.empty_like(x[0]), torch.empty_like(x[1])
    H.h3attn_rotary(rope, pos, x[0], ref_q, x[1], ref_k)
    ref, ref_lse = W.outputs(n, heads)
    with H.Plan(docs_1d([n]), heads) as plan:
        H.h3attn_plan_set_causal(plan.handle, kv)
        H.h3attn_forward_causal(plan.handle, ref_q, ref_k, x[2], ref, W.SCALE, ref_lse)
        torch.cuda.synchronize()
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s), H.Plan(docs_1d([n]), heads) as plan:
                H.h3attn_plan_set_causal(plan.handle, kv)
                for _ in range(20):
                    q2, k2 = torch.zeros_like(ref_q), torch.zeros_like(ref_k)
                    o, lse = W.outputs(n, heads)
                    H.h3attn_rotary(rope, pos, x[0], q2, x[1], k2)
                    H.h3attn_forward_causal(plan.handle, q2, k2, x[2], o, W.SCALE, lse)
                    s.synchronize()
                    if not (torch.equal(q2, ref_q) and torch.equal(o, ref) and torch.equal(lse, ref_lse)):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]

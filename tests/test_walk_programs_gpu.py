"""The sparse and prefix calls as programs make them: first of all inside a
capture, from several host threads with a plan and a stream each, and on a plan
that takes the place of a destroyed one."""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import walks
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d

pytestmark = pytest.mark.gpu

# No kernel of the library has run in the process when the capture begins.
CHILD = """
import numpy as np
import torch
from oracle import walks
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W

s, few, many = W.Sparse([1300, 260], 3, 512, 4), W.Prefix([1] * 9, 3, 700), W.Prefix([300, 900], 3, 700)
q, k, v = (W.rows(1560, 3, i) for i in range(3))
kp, vp = (W.rows(700, 3, 5 + i) for i in range(2))
out = [W.outputs(n, 3) for n in (1560, 9, 1200)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    H.h3attn_block_select(s.plan.handle, W.flat(q), W.flat(k), 4, s.idx, s.cnt)
    s.forward(q, k, v, *out[0])
    few.forward(q[:9], k[:9], v[:9], kp, vp, *out[1])
    many.forward(q[:1200], k[:1200], v[:1200], kp, vp, *out[2])
graph.replay()
torch.cuda.synchronize()
idx, cnt = walks.select(W.f64(q), W.f64(k), s.cu, 512, 4, True)
assert np.array_equal(s.idx.cpu().numpy(), idx)
W.check(*out[0], q, [k], walks.sparse_attention(W.f64(q), W.f64(k), W.f64(v), s.cu, 512, idx, cnt, W.SCALE))
for p, n, (o, lse) in ((few, 9, out[1]), (many, 1200, out[2])):
    t = (q[:n], k[:n], v[:n], kp, vp)
    W.check(o, lse, q[:n], [k[:n], kp], walks.prefix_attention(*(W.f64(x) for x in t), p.cu, W.SCALE))
"""


def test_first_calls_of_a_process_captured(lib):
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


def test_host_threads_with_a_plan_and_a_stream_each(lib):
    errors = []

    def work(seed):
        try:
            rng, stream = np.random.default_rng(seed), torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(8):
                    lens, heads = [int(x) for x in rng.integers(1, 900, rng.integers(1, 5))], int(rng.integers(1, 4))
                    s, prefix = W.Sparse(lens, heads, int(rng.choice([256, 512])), int(rng.integers(1, 8))), int(rng.integers(1, 900))
                    H.h3attn_plan_set_prefix(s.plan.handle, prefix)
                    t = [W.rows(n, heads, int(rng.integers(1 << 30))) for n in (s.S, s.S, s.S, prefix, prefix)]
                    idx, cnt = s.select(t[0], t[1], s.max_blocks)
                    o, lse = s.forward(*t[:3])
                    o2, lse2 = W.outputs(s.S, heads)
                    H.h3attn_forward_prefix(s.plan.handle, *(W.flat(x) for x in t), W.flat(o2), W.SCALE, lse2)
                    W.ok(s.plan)
                    f = [W.f64(x) for x in t]
                    want = walks.select(f[0], f[1], s.cu, s.q_block, s.max_blocks, False)
                    assert np.array_equal(idx, want[0]) and np.array_equal(cnt, want[1])
                    W.check(o, lse, t[0], [t[1]], walks.sparse_attention(*f[:3], s.cu, s.q_block, idx, cnt, W.SCALE))
                    W.check(o2, lse2, t[0], [t[1], t[3]], walks.prefix_attention(*f, s.cu, W.SCALE))
        except BaseException as e:  # reported on the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(seed,)) for seed in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_a_plan_in_a_destroyed_ones_place_has_no_lists(lib):
    # (a new plan may get the old one's address)
    for _ in range(4):
        s = W.Sparse([40], 1, 256, 1)
        H.h3attn_plan_set_prefix(s.plan.handle, 3)
        handle = s.plan.handle
        s.plan.close()
        for known in (H._plan_rows, H._prefix_rows, H._list_sizes, H._plan_device):
            assert handle not in known
        with H.Plan(docs_1d([4000]), 3) as plan:
            t = W.flat(W.rows(4000, 3, 1))
            o = torch.empty_like(t)
            idx = torch.zeros(3, 16, 1, dtype=torch.int32, device="cuda")
            for call in (lambda: H.h3attn_block_select(plan.handle, t, t, 1, idx, idx),
                         lambda: H.h3attn_forward_sparse(plan.handle, t, t, t, idx, idx, o, 0.1),
                         lambda: H.h3attn_forward_prefix(plan.handle, t, t, t, t, t, o, 0.1)):
                with pytest.raises(H.H3AttnError) as e:
                    call()
                assert e.value.status == H.H3ATTN_EINVAL

"""A call that fails in the CUDA runtime leaves nothing behind that a later
call takes for a failure of its own."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# The failing call: adding a list to a plan on a stream that is being captured
# (not allowed, and refused by the runtime).
CHILD = """
import sys
import torch
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W
from tests.gpu_cases import docs_1d

plan = H.Plan(docs_1d([300]), 2)
q, k, v = (W.flat(W.rows(300, 2, i)) for i in range(3))
kp, vp = (W.flat(W.rows(50, 2, 3 + i)) for i in range(2))
o, lse = W.outputs(300, 2)
o = W.flat(o)
H.h3attn_plan_set_prefix(plan.handle, 50)
gq, kout = torch.ones(128, device="cuda"), torch.empty_like(k)
idx = torch.zeros(2, 2, 2, dtype=torch.int32, device="cuda")
cnt = torch.ones(2, 2, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(side):
    graph.capture_begin()
    try:
        H.h3attn_plan_set_sparse(plan.handle, 256, 2, stream=side)
        raise SystemExit("the call was not refused")
    except H.H3AttnError as e:
        assert e.status == H.H3ATTN_ECUDA, e
    try:
        graph.capture_end()
    except RuntimeError:
        pass  # (the runtime ends a capture in which it refused a call)
call = sys.argv[1]
if call == "prefix":
    H.h3attn_forward_prefix(plan.handle, q, k, v, kp, vp, o, W.SCALE, lse, stream=0)
elif call == "dense":
    H.h3attn_forward(plan.handle, q, k, v, o, W.SCALE, lse, stream=0)
elif call == "prologue":
    H.h3attn_qk_prologue(plan.handle, q, k, o, kout, gq, gq, 1e-6, stream=0)
else:
    H.h3attn_plan_set_sparse(plan.handle, 256, 2, stream=0)  # and the refused call itself, again
    info = H.h3attn_plan_sparse_info(plan.handle)
    assert info["n_q_blocks"] == 2
    H.h3attn_block_select(plan.handle, q, k, 2, idx, cnt, stream=0)
"""


@pytest.mark.parametrize("call", ["prefix", "dense", "prologue", "sparse"])
def test_the_next_call_succeeds(lib, call):
    r = subprocess.run([sys.executable, "-c", CHILD, call], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]

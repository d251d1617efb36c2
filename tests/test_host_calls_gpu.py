"""Calls that stay on the host (listings, refusals) do not initialise CUDA: a
process that has made them may still fork ones that use the GPU."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import os
from packed_varlen_non_gb300 import h3attn as H

H.h3attn_walk_list_host(0, [0, 10], 2, 256, 1, 4)
H.h3attn_work_list_host([0, 10], 2, 4)
for fn in (lambda: H.h3attn_plan_info(None), lambda: H.h3attn_forward(None, 16, 16, 16, 16, 0.1, qkv_row_stride=128, o_row_stride=128, stream=0),
           lambda: H.h3attn_walk_list_host(3, [0, 10], 2, 256, 1, 4), lambda: H.h3attn_plan_create([], 2, stream=False)):
    try:
        fn()
        raise SystemExit("not refused")
    except H.H3AttnError:
        pass
H.h3attn_plan_destroy(None)
pid = os.fork()
if pid == 0:
    code = 1
    try:
        with H.Plan([[(5, 1, 1, (0.0, 0.0, 0.0), (1.0, 0.0, 0.0))]], 2, stream=0) as plan:
            H.h3attn_get_device_error(plan.handle, stream=0)
        code = 0
    finally:
        os._exit(code)
raise SystemExit(os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]))
"""


def test_a_process_may_fork_after_host_calls(lib):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", CHILD], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]

"""A call that CUDA refuses reports it, and the next call does not report it again."""
import subprocess
import sys
from pathlib import Path

import pytest

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu

# A capture that a synchronisation has ended takes no launch (an error code, no fault).  In a
# process of its own: PyTorch may go on taking that capture for an open one.
CODE = """
import torch
import paged_kv_cache_301_gb300 as pa
B, H, D, bs = 4, 2, 64, 16
half = dict(dtype=torch.float16, device="cuda")
q, k, v, out = (torch.ones(B, H, D, **half) for _ in range(4))
kp, vp = torch.zeros(8, bs, H, D, **half), torch.zeros(8, bs, H, D, **half)
tables = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
lens = torch.ones(B, dtype=torch.int32, device="cuda")
k8 = pa.alloc_cache_q8(8, H, bs, D)
refused = {
    "pa_rope_append": lambda: pa.pa_rope_append(out, kp, vp, q, k, v, None, tables, lens),
    "pa_rope_append_q8": lambda: pa.pa_rope_append_q8(out, *k8, q, k, v, None, tables, lens),
    "pa_decode_q8": lambda: pa.pa_decode_q8(out, q, *k8, tables, lens, 0.1, workspace=ws8),
    "pa_expand_blocks_q8": lambda: pa.pa_expand_blocks_q8(kp, vp, *k8, pairs),
    "pa_append_tokens": lambda: pa.pa_append_tokens(kp, vp, k, v, tables, lens),
}["%s"]
pairs = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
ws, ws8 = pa.workspace_for(q, kp, tables, bs), pa.workspace_for_q8(q, k8[0], bs)
refused()
pa.set_decode_path("simt")
pa.pa_decode(out, q, kp, vp, tables, lens, 0.1, workspace=ws)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(torch.cuda.Stream()):
    graph.capture_begin(capture_error_mode="global")
    try:
        torch.cuda.synchronize()
    except RuntimeError:
        pass
    try:
        refused()
        raise SystemExit("the call was taken")
    except pa.PagedAttnError as e:
        assert e.status == 4
    try:
        graph.capture_end()
    except RuntimeError:
        pass
for _ in range(2):
    pa.pa_decode(out, q, kp, vp, tables, lens, 0.1, workspace=ws)
torch.cuda.synchronize()
print("done", flush=True)
"""


@pytest.mark.parametrize("call", ["pa_rope_append", "pa_rope_append_q8", "pa_decode_q8",
                                  "pa_expand_blocks_q8", "pa_append_tokens"])
def test_a_refused_launch_is_reported_once(call):
    lib()
    run = subprocess.run([sys.executable, "-c", CODE % call], capture_output=True, text=True,
                         timeout=120, cwd=Path(__file__).resolve().parent.parent)
    assert run.returncode == 0 and "done" in run.stdout, run.stdout + run.stderr

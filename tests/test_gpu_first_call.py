"""A call of a process may be its first and be captured into a graph at once."""
import subprocess
import sys
from pathlib import Path

import pytest

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu

CODE = """
import torch
import paged_kv_cache_301_gb300 as pa
B, H, G, D, bs, n = 3, 2, 4, 128, 16, 1600
g = torch.Generator("cuda").manual_seed(3)
rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
NB = B * n // bs
tables = torch.randperm(NB, generator=g, device="cuda").to(torch.int32).view(B, -1)
lens, starts = i32([n] * B), i32([0, n, 2 * n, 3 * n])
T = B * n
cs = pa.rope_table(n, D)
c8 = pa.alloc_cache_q8(NB, H, bs, D)
k16, v16 = (torch.zeros(NB, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
q, k, v, w = rand(T, H * G, D), rand(T, H, D), rand(T, H, D), rand(D)
q1, k1, v1 = rand(B, H * G, D), rand(B, H, D), rand(B, H, D)
qo, o1 = torch.empty_like(q), torch.zeros_like(q1)
ws = pa.workspace_for_q8(q1, c8[0], n)
for x in c8[:2]:
    x.copy_(torch.randn(NB, H, bs, D, generator=g, device="cuda").to(pa.E4M3))
pairs = torch.arange(NB, dtype=torch.int32, device="cuda")[:, None].expand(NB, 2).contiguous()
call, results = {
    "prompts": (lambda: pa.pa_rope_append(qo, k16, v16, q, k, v, cs, tables, lens, q_start=starts,
                                          q_weight=w), [qo, k16, v16]),
    "step": (lambda: pa.pa_rope_append(o1, k16, v16, q1, k1, v1, cs, tables, lens), [o1, k16]),
    "prompts8": (lambda: pa.pa_rope_append_q8(qo, *c8, q, k, v, cs, tables, lens, q_start=starts),
                 [qo, *c8]),
    "step8": (lambda: pa.pa_rope_append_q8(o1, *c8, q1, k1, v1, cs, tables, lens), [o1, *c8]),
    "decode8": (lambda: pa.pa_decode_q8(o1, q1, *c8, tables, lens, 0.1, max_seq_len=n,
                                        workspace=ws), [o1]),
    "decode8 alloc": (lambda: pa.pa_decode_q8(o1, q1, *c8, tables, lens, 0.1, max_seq_len=n), [o1]),
    "expand8": (lambda: pa.pa_expand_blocks_q8(k16, v16, *c8, pairs), [k16, v16]),
}["%s"]
before = [r.clone() for r in results]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = [r.clone() for r in results]
for r, b in zip(results, before):
    r.copy_(b)
call()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, results))
assert any(not torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, before))
print("done", flush=True)
"""


@pytest.mark.parametrize("call", ["prompts", "step", "prompts8", "step8", "decode8",
                                  "decode8 alloc", "expand8"])
def test_a_first_call_is_captured(call):
    lib()
    run = subprocess.run([sys.executable, "-c", CODE % call], capture_output=True, text=True,
                         timeout=120, cwd=Path(__file__).resolve().parent.parent)
    assert run.returncode == 0 and "done" in run.stdout, run.stdout + run.stderr

"""The first call of a process of the latent cache and of drafted trees may be captured into a
graph at once."""
import subprocess
import sys
from pathlib import Path

import pytest

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu

CODE = """
import torch
import paged_kv_cache_301_gb300 as pa
B, H, G, D, R, bs, n = 3, 2, 4, 128, 512, 16, 1600
g = torch.Generator("cuda").manual_seed(3)
rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
NB = B * n // bs
tables = torch.randperm(NB, generator=g, device="cuda").to(torch.int32).view(B, -1)
lens, new, every = i32([n] * B), i32([0, 5, 8, 20]), i32([0, n, 2 * n, 3 * n])
T = 20
k16, v16, pool = rand(NB, bs, H, D), rand(NB, bs, H, D), rand(NB, bs, R + 64)
q, ql, x = rand(T, H * G, D), rand(T, 16, R + 64), rand(T, R + 64)
o, ol, rows = torch.zeros_like(q), torch.zeros_like(ql[..., :R]), rand(B * n, R + 64)
qr, qo = rand(T, 16, 64), torch.zeros(T, 16, 64, dtype=torch.bfloat16, device="cuda")
qe, kv = rand(T, 4, 192), rand(B * n, 4, 256)
oe = torch.zeros(T, 4, 128, dtype=torch.bfloat16, device="cuda")
cs = pa.rope_table(n, 64)
ws, wl = pa.workspace_for_tree(q, k16, 12), pa.workspace_for_latent(ol, pool, 12)
kw = dict(max_q_len=12, max_seq_len=n)
call, results = {
    "tree": (lambda: pa.pa_decode_tree(o, q, k16, v16, tables, lens, new, 0.1, workspace=ws, **kw),
             [o]),
    "tree alloc": (lambda: pa.pa_decode_tree(o, q, k16, v16, tables, lens, new, 0.1, **kw), [o]),
    "latent": (lambda: pa.pa_latent_decode(ol, ql, pool, tables, lens, 0.1, q_start=new,
                                           workspace=wl, **kw), [ol]),
    "append": (lambda: pa.pa_latent_append(pool, x[:, :R], x[:, R:], cs, tables, lens, q_start=new,
                                           q_rope=qr, q_out=qo), [pool, qo]),
    "gather": (lambda: pa.pa_latent_gather(rows, pool, tables, lens, every), [rows]),
    "prefill": (lambda: pa.pa_latent_prefill(oe, qe, kv, rows[:, R:], new, every, 0.1,
                                             max_q_len=12), [oe]),
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
bits = lambda t: t.contiguous().view(torch.uint8)
assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, results))
assert all(not torch.equal(bits(a), bits(b)) for a, b in zip(got, before))
print("done", flush=True)
"""


@pytest.mark.parametrize("call", ["tree", "tree alloc", "latent", "append", "gather", "prefill"])
def test_a_first_call_is_captured(call):
    lib()
    run = subprocess.run([sys.executable, "-c", CODE % call], capture_output=True, text=True,
                         timeout=120, cwd=Path(__file__).resolve().parent.parent)
    assert run.returncode == 0 and "done" in run.stdout, run.stdout + run.stderr

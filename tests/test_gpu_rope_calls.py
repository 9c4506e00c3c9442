"""Rotated cache writes called from several host threads at once."""
import threading

import pytest
import torch

from tests.gpu_helpers import i32, lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_two_threads_with_two_shapes_of_one_kernel(q8):
    """Two threads write prompts of one type and head_dim, whose CTAs need different
    amounts of shared memory (77 KB and 43 KB): every call is taken.  Through the C entry,
    which holds no lock of Python's."""
    pa = lib()
    f = pa.lib().pa_rope_append_q8 if q8 else pa.lib().pa_rope_append
    D, bs, T, NB = 128, 16, 2432, 152
    jobs = []
    for Hq, H, R in ((32, 8, 128), (20, 4, 16)) if not q8 else ((64, 8, 128), (12, 8, 16)):
        g = torch.Generator("cuda").manual_seed(Hq)
        q, k, v = (torch.randn(T, n, D, generator=g, device="cuda").to(torch.bfloat16)
                   for n in (Hq, H, H))
        table = pa.rope_table(T, R)
        out = torch.empty_like(q)
        if q8:
            pools = pa.alloc_cache_q8(NB, H, bs, D)
        else:
            pools = [torch.zeros(NB, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        tables = torch.arange(NB, dtype=torch.int32, device="cuda")[None].contiguous()
        held = (out, *pools, q, k, v, table, tables, i32([T]), i32([0, T]))
        p = [t.data_ptr() for t in held]
        n = 1 + len(pools)
        s = torch.cuda.Stream()
        jobs.append((held, s, (*p[:n], *p[n:n + 3], None, None, 1e-6, p[n + 3], T, R, 0, None,
                               *p[n + 4:], 1, T, 0, 0, Hq, H, D, bs, NB, NB, 1, None,
                               s.cuda_stream)))
    torch.cuda.synchronize()
    start, got = threading.Barrier(2), [[], []]

    def work(i):
        start.wait()
        for _ in range(3000):
            got[i].append(f(*jobs[i][2]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [sum(x != 0 for x in g) for g in got] == [0, 0]

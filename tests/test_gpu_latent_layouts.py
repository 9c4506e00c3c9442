"""pa_latent_append's queries in place and beside its inputs, as parts of the same rows: the bits
of calls with tensors of their own."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import i32, lib
from tests.paged_rows import Pages, starts

pytestmark = pytest.mark.gpu
P, R = 64, 256


@pytest.fixture(scope="module")
def pa():
    return lib()


def call(pa, p, pool, lat, key, q, out, lens, counts):
    pa.pa_latent_append(pool, lat, key, pa.rope_table(max(lens), P), i32(p.tables), i32(lens),
                        q_start=i32(starts(counts)), q_rope=q, q_out=out)


@pytest.mark.parametrize("counts", [[40], [1]])
def test_the_same_object_twice(pa, counts):
    """q_rope and q_out one Python object, a part of wider rows."""
    g = np.random.default_rng(8)
    p = Pages([40], 16, g)
    pool = p.pool((R + P,), torch.float16, g)
    T = counts[0]
    wide = torch.from_numpy(g.normal(size=(T, 3, 3 * P))).half().cuda()
    y = torch.from_numpy(g.normal(size=(T, R + P))).half().cuda()
    before, want = wide.clone(), torch.empty(T, 3, P, dtype=wide.dtype, device="cuda")
    q = wide[..., P:2 * P]
    call(pa, p, pool, y[:, :R], y[:, R:], q.clone(), want, [40], counts)
    call(pa, p, pool, y[:, :R], y[:, R:], q, q, [40], counts)
    before[..., P:2 * P] = want
    assert torch.equal(wide, before)

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


def parts_of(x, H, layout):
    """latent, key, q, q_out as views of x [T, width]."""
    T = x.shape[0]
    if layout == "in place":                      # [q heads | latent | key]
        q = x[:, :H * P].view(T, H, P)
        return x[:, H * P:H * P + R], x[:, H * P + R:H * P + R + P], q, q
    if layout == "beside":                        # [q heads, each with room behind it | ...]
        q = x[:, :H * 2 * P].view(T, H, 2 * P)
        at = H * 2 * P
        return x[:, at:at + R], x[:, at + R:at + R + P], q[..., :P], q[..., P:]
    # [q heads | latent | key | absorbed queries, the rotated part last]
    at = H * P + R + P
    wide = x[:, at:at + H * (R + P)].view(T, H, R + P)
    return x[:, H * P:H * P + R], x[:, H * P + R:at], x[:, :H * P].view(T, H, P), wide[..., R:]


@pytest.mark.parametrize("layout", ["in place", "beside", "apart"])
@pytest.mark.parametrize("H", [1, 2, 17])
@pytest.mark.parametrize("lens,counts", [([30, 9], [30, 5]), ([20], [1])])
def test_parts_of_one_projection(pa, layout, H, lens, counts):
    g = np.random.default_rng(H)
    p = Pages(lens, 16, g)
    T, width = sum(counts), {"in place": H * P, "beside": 2 * H * P,
                             "apart": H * P + H * (R + P)}[layout] + R + P + 8
    x = torch.from_numpy(g.normal(size=(T, width))).bfloat16().cuda()
    pool = p.pool((R + P,), torch.bfloat16, g)
    want_pool, before = pool.clone(), x.clone()
    lat, key, q, out = parts_of(x, H, layout)
    want = torch.empty(T, H, P, dtype=x.dtype, device="cuda")
    call(pa, p, want_pool, lat.clone(), key.clone(), q.clone(), want, lens, counts)
    call(pa, p, pool, lat, key, q, out, lens, counts)
    assert torch.equal(out, want) and not torch.equal(want, before[:, :H * P].view(T, H, P))
    assert torch.equal(pool.view(torch.int16), want_pool.view(torch.int16))
    out.zero_()
    a = parts_of(before, H, layout)[3]
    a.zero_()
    assert torch.equal(x, before)                 # and nothing else of the rows


def test_one_head_beside_itself(pa):
    """q and q_out are the halves of x [T, 1, 128]."""
    g = np.random.default_rng(7)
    p = Pages([40], 16, g)
    pool = p.pool((R + P,), torch.float16, g)
    x = torch.from_numpy(g.normal(size=(40, 1, 2 * P))).half().cuda()
    y = torch.from_numpy(g.normal(size=(40, R + P))).half().cuda()
    want = torch.empty(40, 1, P, dtype=x.dtype, device="cuda")
    call(pa, p, pool, y[:, :R], y[:, R:], x[..., :P].clone(), want, [40], [40])
    call(pa, p, pool, y[:, :R], y[:, R:], x[..., :P], x[..., P:], [40], [40])
    assert torch.equal(x[..., P:], want)
    with pytest.raises(pa.PagedAttnError):
        call(pa, p, pool, y[:, :R], y[:, R:], x[..., :P], x[..., 32:32 + P], [40], [40])


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

"""Block moves of the latent cache by the calls that move blocks of any pool: copy-on-write of
every layer's pool at once, and swaps to pinned memory and back."""
import torch
import pytest

from tests.gpu_helpers import i32, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return lib()


def pools(n, NB, bs, R, dt, **kw):
    return [torch.randn(NB, bs, R + 64, **kw).to(dt) for _ in range(n)]


@pytest.mark.parametrize("bs,R,dt", [(8, 256, torch.float16), (16, 512, torch.bfloat16)])
def test_copy_blocks(pa, bs, R, dt):
    layers = pools(3, 9, bs, R, dt, device="cuda")
    want = [x.clone() for x in layers]
    for x in want:
        x[7], x[2] = x[0], x[5]
    pa.pa_copy_blocks_multi(layers, i32([[0, 7], [5, 2]]))
    assert all(torch.equal(a, b) for a, b in zip(layers, want))


@pytest.mark.parametrize("bs,R,dt", [(8, 256, torch.float16), (64, 512, torch.bfloat16)])
def test_swap_blocks(pa, bs, R, dt):
    layers = pools(2, 6, bs, R, dt, device="cuda")
    host = [torch.zeros(4, bs, R + 64, dtype=dt).pin_memory() for _ in layers]
    pa.pa_swap_blocks(host, layers, i32([[5, 0], [1, 3]]))
    torch.cuda.synchronize()
    for x, h in zip(layers, host):
        assert torch.equal(h[0], x[5].cpu()) and torch.equal(h[3], x[1].cpu())
        assert not h[1:3].any()
    pa.pa_swap_blocks(layers, host, i32([[3, 4]]))
    torch.cuda.synchronize()
    assert all(torch.equal(x[4], x[1]) for x in layers)

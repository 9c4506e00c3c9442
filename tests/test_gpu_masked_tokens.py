"""A single new token whose set leaves itself out: its values have no part in its row, whatever
they are.  Against the fp64 definition (bounds: tests/paged_rows.py)."""
import pytest
import torch

from tests import test_gpu_latent as latent
from tests import test_gpu_tree as tree
from tests.gpu_helpers import i32, lib
from tests.paged_rows import f64

pytestmark = pytest.mark.gpu
LENS = [300, 1, 128, 65, 17]
OUT = [0, 1, 2, 4]                  # the sequences whose new token is left out


@pytest.fixture(scope="module")
def pa():
    return lib()


def leave_out(b, pool, x):
    """Their bits cleared, and `x` in one element of their values."""
    for s in OUT:
        b.mask[s] = 0
        t = b.lens[s] - 1
        pool[b.p.tables[s, t // b.p.bs], t % b.p.bs, ..., 40] = x
    return b


@pytest.mark.parametrize("x", [float("inf"), float("nan")])
@pytest.mark.parametrize("starts", [True, False])
@pytest.mark.parametrize("D,G,dt", [(64, 1, "fp16"), (128, 4, "bf16"), (128, 40, "bf16")])
def test_tree(pa, D, G, dt, starts, x):
    b = tree.Batch(LENS, [1] * 5, 2 * G, 2, D, 16, dt)
    leave_out(b, b.v, x)
    if starts:
        b.run(pa)
    else:
        pa.pa_decode_tree(b.out, b.q, b.k, b.v, i32(b.p.tables), i32(LENS), None, b.scale,
                          tree_mask=i32(b.mask))
    b.check()
    assert (f64(b.out)[1] == 0).all()


@pytest.mark.parametrize("x", [float("inf"), float("nan")])
@pytest.mark.parametrize("starts", [True, False])
@pytest.mark.parametrize("R,H,dt", [(256, 3, "fp16"), (512, 16, "bf16"), (512, 70, "bf16")])
def test_latent(pa, R, H, dt, starts, x):
    b = latent.Batch(LENS, [1] * 5, H, R, 16, dt)
    leave_out(b, b.pool, x)
    if not starts:
        b.q_start = None
    b.run(pa).check(heads=sorted({0, H // 2, H - 1}))
    assert (f64(b.out)[1] == 0).all()
    assert torch.isfinite(b.out).all()

"""two_terms: the softmax weights in two terms of the storage type, whatever the shape.  Against
the fp64 definitions, bounds for two terms (tests/paged_rows.py)."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from tests import test_gpu_latent as latent
from tests import test_gpu_tree as tree
from tests.gpu_helpers import i32, lib
from tests.paged_rows import assert_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return lib()


def two(b, pa, **kw):
    b.terms = 2
    return b.run(pa, two_terms=True, **kw)


@pytest.mark.parametrize("case", [
    ([1, 2, 3, 40], [1, 2, 3, 4], 128, 1, 128, 16, "bf16", "tree"),
    ([17, 64, 65, 128, 129], [5, 1, 16, 7, 9], 16, 2, 128, 16, "fp16", "tree"),
    ([300, 40, 1000], [33, 40, 64], 8, 2, 128, 32, "bf16", "tree"),
    ([700, 90], [70, 90], 3, 1, 64, 8, "bf16", "star"),
    ([260, 515], [12, 3], 40, 8, 64, 64, "fp16", "causal"),
    ([5, 6], [1, 2], 10, 2, 64, 16, "bf16", "chain"),            # no more than 32 columns
], ids=lambda c: f"{c[2]}-{c[3]}x{c[4]}-{c[6]}-{c[7]}")
def test_tree(pa, case):
    two(tree.Batch(*case), pa).check()


@pytest.mark.parametrize("D,dt", [(64, "bf16"), (128, "fp16")])
def test_tree_split_over_the_length(pa, D, dt):
    two(tree.Batch([6000, 3, 9001, 150], [20, 3, 2, 20], 8, 2, D, 16, dt), pa).check()


def test_tree_unseen_values_have_no_part(pa):
    b = tree.Batch([70, 150, 6], [6, 20, 6], 16, 2, 128, 16, "bf16", "star")
    for s, i, pool, x in ((0, 1, b.v, float("inf")), (1, 3, b.v, float("nan")),
                          (1, 17, b.k, float("nan")), (2, 4, b.k, float("inf"))):
        t = b.lens[s] - b.counts[s] + i
        pool[b.p.tables[s, t // 16], t % 16, 1, 5 * i] = x
    two(b, pa).check()


@pytest.mark.parametrize("case", [
    ([1, 2, 0, 40], [1] * 4, 128, 512, 16, "bf16", "one"),
    ([63, 128, 129, 700], [1] * 4, 128, 256, 64, "fp16", "one"),
    ([70, 300, 9], [3, 1, 9], 16, 512, 64, "bf16", "tree"),
    ([200, 7], [2, 1], 70, 256, 16, "bf16", "star"),
    ([140, 90], [80, 66], 3, 512, 16, "fp16", "star"),
], ids=lambda c: f"{c[2]}x{c[3]}-{c[5]}-{c[6]}")
def test_latent(pa, case):
    b = latent.Batch(*case)
    two(b, pa).check(heads=sorted({0, b.H // 2, b.H - 1}))


def test_latent_split_over_the_length(pa):
    b = latent.Batch([4000, 3, 9001, 150], [1] * 4, 128, 512, 16, "bf16", "one")
    ws = pa.workspace_for_latent(b.out, b.pool)                  # that of one term is enough
    two(b, pa, workspace=ws).check(heads=[0, 64, 127])


class Prompts(latent.Prompts):
    def check2(self, heads=None):
        got, q, kv, k = f64(self.out), f64(self.q), f64(self.kv), f64(self.k)
        for b, (L, n) in enumerate(zip(self.lens, self.counts)):
            mine, rows = slice(self.qs[b], self.qs[b] + n), slice(self.ks[b], self.ks[b] + L)
            for h in heads or range(self.H):
                key = np.concatenate([kv[rows, h, :128], k[rows]], 1)
                ref = ol.attend(q[mine, h], key, kv[rows, h, 128:], ol.visible(n, L), self.scale)
                assert_rows(got[mine, h], *ref, 192, self.dt, 2, (b, h))


@pytest.mark.parametrize("lens,counts,H,dt", [
    ([1, 2, 3], [1, 2, 3], 3, "fp16"),
    ([5, 128, 129], [5, 128, 129], 3, "bf16"),
    ([127, 300, 64], [127, 300, 64], 4, "fp16"),
    ([700, 33], [130, 1], 2, "bf16"),
    ([640, 0, 90], [255, 0, 90], 1, "bf16"),
])
def test_prefill(pa, lens, counts, H, dt):
    Prompts(lens, counts, H, dt).run(pa, two_terms=True).check2()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_prefill_scores_far_apart(pa, dt):
    b = Prompts([900], [900], 2, dt)
    b.kv[::97, :, :128] *= torch.linspace(1, 30, 10, device="cuda", dtype=b.dt)[:, None, None]
    b.run(pa, two_terms=True).check2()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_prefill_unseen_tokens_have_no_part(pa, dt):
    b = Prompts([300, 140], [300, 140], 2, dt)
    b.kv[200, 0, 130] = float("inf")
    b.kv[7, 1, 190] = float("-inf")
    b.kv[250, 1, 3] = float("nan")
    b.kv[300, 1, 200] = float("nan")                  # the next sequence's first token
    b.k[300 + 77, 5] = float("inf")
    b.run(pa, two_terms=True).check2()


def test_a_chain_as_prefill_has_it(pa):
    """A drafted chain of 64 columns: both calls within the bound of two terms of one definition."""
    b = tree.Batch([3, 40, 300], [3, 16, 16], 8, 2, 128, 16, "bf16", "causal")
    two(b, pa).check()
    b.out.fill_(7.0)
    pa.pa_prefill(b.out, b.q, b.k, b.v, i32(b.p.tables), i32(b.lens), i32(b.starts), b.scale)
    b.check()

"""Drafted trees of more new tokens than a tile of the cache holds (64 tokens at latent 512, else
128): a row may see nothing of the tile that its part of the work begins with, and its first
tokens in a later one.  Against the fp64 definition (bounds: tests/paged_rows.py)."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from tests import test_gpu_latent as latent
from tests import test_gpu_tree as tree
from tests.gpu_helpers import lib
from tests.paged_rows import assert_rows, f64, words_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return lib()


def parents_of(n, kind, g):
    """star: each token hangs on the context; branches: chains of eight do; tree: on any."""
    if kind == "star":
        return [-1] * n
    if kind == "branches":
        return [i - 1 if i % 8 else -1 for i in range(n)]
    return [int(g.integers(-1, i)) if i else -1 for i in range(n)]


def hang(b, kind):
    g = np.random.default_rng(sum(b.lens))
    b.mask = np.concatenate([words_of(parents_of(n, kind, g), b.W) for n in b.counts])
    return b


class Latent(latent.Batch):
    def check(self):
        super().check(heads=sorted({0, self.H // 2, self.H - 1}))


LATENT = [
    # lens, new tokens, heads, latent, block: contexts of whole tiles, of an odd rest, of none
    ([720], [80], 16, 512, 16),
    ([840], [200], 16, 512, 64),
    ([66], [66], 16, 512, 8),
    ([80, 1003, 333], [80, 200, 66], 5, 512, 16),
    ([386], [130], 16, 256, 16),
    ([300], [300], 8, 256, 32),
    ([811, 131], [300, 130], 4, 256, 16),
    ([3000], [100], 8, 512, 16),
]
TREE = [
    # lens, new tokens, query heads, KV heads, head_dim, block
    ([386], [130], 8, 2, 128, 16),
    ([300], [300], 4, 1, 128, 16),
    ([811, 131], [300, 130], 8, 4, 64, 32),
    ([556], [300], 5, 1, 64, 8),
    ([130], [130], 16, 2, 64, 16),
    ([3000], [150], 4, 1, 128, 16),
]


@pytest.mark.parametrize("kind", ["branches", "star", "tree"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", LATENT, ids=lambda c: f"{c[3]}-{c[0][0]}-{c[1][0]}")
def test_latent(pa, case, dt, kind):
    hang(Latent(*case, dt), kind).run(pa).check()


@pytest.mark.parametrize("kind", ["branches", "star", "tree"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", TREE, ids=lambda c: f"{c[4]}-{c[0][0]}-{c[1][0]}")
def test_tree(pa, case, dt, kind):
    hang(tree.Batch(*case, dt), kind).run(pa).check()


def lower(b, pools, dim, by):
    """Every score is lower by `by` in base 2: q is 4 at `dim`, and the keys what makes it so."""
    b.q[..., dim] = 4
    for x in pools:
        live = torch.from_numpy(b.p.live).to(x.device)
        x[live, ..., dim] = -by / (4 * b.scale * 1.4426950408889634)


@pytest.mark.parametrize("n,L", [(200, 200), (200, 300), (80, 720)])
def test_latent_low_scores(pa, n, L):
    """Weights against any reference but the row's own maximum have no bits left in fp16."""
    b = hang(Latent([L], [n], 16, 512, 16, "fp16"), "branches")
    lower(b, [b.pool], 512 + 7, 40)
    b.run(pa).check()


@pytest.mark.parametrize("n,L", [(300, 300), (300, 411), (130, 386)])
def test_tree_low_scores(pa, n, L):
    b = hang(tree.Batch([L], [n], 8, 2, 128, 16, "fp16"), "branches")
    lower(b, [b.k], 7, 40)
    b.run(pa).check()


def check_without(b, first, heads, rows_of, Dk):
    """Against attention over the tokens from `first` on: older ones have a weight of zero."""
    got, q = f64(b.out), f64(b.q)
    seen = ol.visible(b.counts[0], b.lens[0], b.mask)[:, first:]
    for h in heads:
        k, v = rows_of(h)
        ref = ol.attend(q[:, h], k[first:], v[first:], seen, b.scale)
        assert_rows(got[:, h], *ref, Dk, b.dt, b.terms, h)


@pytest.mark.parametrize("L,n", [(500, 5), (700, 200)])
def test_tree_first_tiles_of_no_weight(pa, L, n):
    """Scores of -inf in all of the first tiles, low ones behind them."""
    b = hang(tree.Batch([L], [n], 8, 2, 64, 16, "fp16"), "branches")
    lower(b, [b.k], 7, 40)
    for t in range(256):
        b.k[b.p.tables[0, t // 16], t % 16, :, 7] = -float("inf")
    b.run(pa)
    k, v = b.p.rows(f64(b.k), 0), b.p.rows(f64(b.v), 0)
    check_without(b, 256, range(8), lambda h: (k[:, h // 4], v[:, h // 4]), 64)


@pytest.mark.parametrize("L,n", [(400, 5), (420, 100)])
def test_latent_first_tiles_of_no_weight(pa, L, n):
    b = hang(Latent([L], [n], 16, 512, 16, "fp16"), "branches")
    lower(b, [b.pool], 512 + 7, 40)
    for t in range(128):
        b.pool[b.p.tables[0, t // 16], t % 16, 512 + 7] = -float("inf")
    b.run(pa)
    x = b.p.rows(f64(b.pool), 0)
    check_without(b, 128, [0, 15], lambda h: (x, x[:, :512]), 576)


def test_many_wide_trees(pa):
    """More items than CTAs, so that windows begin anywhere among the new tokens."""
    g = np.random.default_rng(4)
    counts = [int(x) for x in g.integers(100, 300, size=24)]
    lens = [n + int(x) for n, x in zip(counts, g.integers(0, 300, size=24))]
    b = hang(Latent(lens, counts, 3, 512, 16, "bf16"), "branches")
    b.run(pa).check()

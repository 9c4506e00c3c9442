"""GPU parity of pa_decode_tree against the fp64 definition (bounds: tests/paged_rows.py)."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from tests.gpu_helpers import i32, lib
from tests.paged_rows import DT, Pages, assert_rows, chain_or_tree, f64, starts, words_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return lib()


class Batch:
    def __init__(self, lens, counts, Hq, H, D, bs, dt, kind="tree", seed=0, W=None, size=1.0):
        g = np.random.default_rng(seed + 100 * D + bs)
        self.lens, self.counts, self.Hq, self.H, self.D, self.dt = lens, counts, Hq, H, D, DT[dt]
        self.p = Pages(lens, bs, g)
        self.k, self.v = (self.p.pool((H, D), self.dt, g, size) for _ in "kv")
        self.T = sum(counts)
        self.q = torch.from_numpy(g.normal(size=(self.T, Hq, D))).to(self.dt).cuda()
        self.out = torch.full((self.T, Hq, D), 7.0, dtype=self.dt, device="cuda")
        self.starts = starts(counts)
        most = max(counts + [1])
        self.W = W or -(-most // 32)
        self.mask = None
        if kind != "causal":
            self.mask = np.concatenate([words_of(chain_or_tree(n, kind, g), self.W)
                                        for n in counts if n] or [np.zeros((0, self.W), np.int32)])
        self.scale = D ** -0.5
        self.terms = 2 if max(counts + [1]) * (Hq // H) <= 32 else 1

    def args(self):
        return (self.out, self.q, self.k, self.v, i32(self.p.tables), i32(self.lens),
                i32(self.starts), self.scale)

    def run(self, pa, **kw):
        if self.mask is not None:
            kw.setdefault("tree_mask", i32(self.mask))
        kw.setdefault("max_q_len", max(self.counts + [0]))
        kw.setdefault("max_seq_len", max(self.lens + [0]))
        pa.pa_decode_tree(*self.args(), **kw)
        return self

    def check(self, skip=()):
        got, q, k, v = f64(self.out), f64(self.q), f64(self.k), f64(self.v)
        G = self.Hq // self.H
        for b, (L, n) in enumerate(zip(self.lens, self.counts)):
            mine = slice(self.starts[b], self.starts[b] + n)
            if b in skip:
                assert (got[mine] == 7.0).all(), b
                continue
            if n == 0:
                continue
            seen = ol.visible(n, L, None if self.mask is None else self.mask[mine])
            kb, vb = self.p.rows(k, b), self.p.rows(v, b)
            for hq in range(self.Hq):
                ref = ol.attend(q[mine, hq], kb[:, hq // G], vb[:, hq // G], seen, self.scale)
                assert_rows(got[mine, hq], *ref, self.D, self.dt, self.terms, (b, hq))


CASES = [
    # lens, new tokens, Hq, H, D, bs, type, what they hang on
    ([1], [1], 1, 1, 64, 8, "fp16", "tree"),
    ([1, 2, 3], [1, 2, 3], 4, 2, 128, 16, "bf16", "tree"),
    ([17, 64, 65, 128, 129], [5, 1, 16, 7, 9], 8, 2, 128, 16, "bf16", "tree"),
    ([127, 128, 129, 255, 300], [4, 4, 4, 4, 4], 4, 4, 64, 16, "fp16", "tree"),
    ([300, 40, 1000], [33, 40, 64], 8, 2, 128, 32, "bf16", "tree"),
    ([700, 90], [70, 90], 3, 1, 64, 8, "bf16", "tree"),
    ([260, 515], [12, 3], 40, 8, 128, 64, "fp16", "chain"),
    ([260, 515], [12, 3], 40, 8, 128, 64, "fp16", "causal"),
    ([511, 77], [31, 32], 16, 1, 128, 16, "bf16", "star"),
    ([2000], [5], 64, 2, 128, 16, "bf16", "tree"),
    ([200, 131], [130, 131], 14, 2, 128, 16, "fp16", "causal"),
    ([100, 0, 50], [3, 0, 4], 6, 2, 64, 16, "bf16", "tree"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[2]}-{c[3]}x{c[4]}-{c[6]}-{c[7]}")
def test_parity(pa, case):
    Batch(*case).run(pa).check()


@pytest.mark.parametrize("D", [64, 128])
def test_split_over_the_length(pa, D):
    """Long sequences are cut between CTAs and joined; short ones stand beside them."""
    Batch([9000, 3, 20001, 150], [7, 3, 2, 20], 8, 2, D, 16, "bf16").run(pa).check()


def test_many_sequences(pa):
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(1, 200, size=400)]
    counts = [int(min(n, x)) for n, x in zip(lens, g.integers(0, 9, size=400))]
    Batch(lens, counts, 4, 2, 128, 16, "bf16").run(pa).check()


def test_one_token_each_without_q_start(pa):
    """q_start None is one token a sequence; an empty sequence's row becomes zeros."""
    lens = [5, 0, 130, 1, 0]
    b = Batch(lens, [1] * 5, 8, 2, 128, 16, "bf16", "causal")
    pa.pa_decode_tree(b.out, b.q, b.k, b.v, i32(b.p.tables), i32(lens), None, b.scale)
    got = f64(b.out)
    assert (got[[1, 4]] == 0).all()
    want = torch.empty_like(b.q)
    pa.pa_decode(want, b.q, b.k, b.v, i32(b.p.tables), i32(lens), b.scale)
    assert (got[[1, 4]] == f64(want)[[1, 4]]).all()
    b.lens, b.counts = [5, 130, 1], [1] * 3
    b.out, b.q = b.out[[0, 2, 3]], b.q[[0, 2, 3]]
    b.p.lens, b.p.tables, b.starts = b.lens, b.p.tables[[0, 2, 3]], starts(b.counts)
    b.check()


def test_rows_that_see_nothing(pa):
    """An empty set with no older token gives zeros; with older ones, those alone."""
    b = Batch([6, 40], [6, 6], 8, 2, 128, 16, "bf16")
    b.mask[2] = 0
    b.mask[8] = 0
    b.run(pa).check()
    assert (f64(b.out)[2] == 0).all()


@pytest.mark.parametrize("D,dt", [(64, "bf16"), (128, "fp16")])
def test_scores_far_apart(pa, D, dt):
    """Maxima that rise from tile to tile, and scores whose weights vanish."""
    b = Batch([1500, 300], [4, 9], 4, 2, D, 16, dt, size=1.0)
    k = b.k.clone()
    for s in range(2):
        for t in range(b.lens[s]):
            if t % 97 == 0:
                k[b.p.tables[s, t // 16], t % 16] *= 1 + t / 40
    b.k = k
    b.run(pa).check()


def test_unseen_values_have_no_part(pa):
    """Infinities and NaN in a drafted token's K and V reach the rows that see it, no others."""
    b = Batch([70, 150, 6], [6, 20, 6], 4, 2, 128, 16, "bf16", "star")
    for s, i, pool, x in ((0, 1, b.v, float("inf")), (1, 3, b.v, float("nan")),
                          (1, 17, b.k, float("nan")), (1, 19, b.v, float("-inf")),
                          (2, 4, b.k, float("inf"))):
        t = b.lens[s] - b.counts[s] + i
        pool[b.p.tables[s, t // 16], t % 16, 1, 5 * i] = x
    b.run(pa).check()


def test_bad_sequences_are_skipped(pa):
    b = Batch([40, 50, 60, 70], [4, 5, 6, 7], 8, 2, 128, 16, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.run(pa, max_q_len=6, status=status)
    assert int(status) == 5
    b.check(skip=(3,))
    b.out.fill_(7.0)
    status.zero_()
    b.run(pa, max_seq_len=55, status=status)
    assert int(status) == 5
    b.check(skip=(2, 3))
    b.out.fill_(7.0)
    lens = i32([3, 50, 10 ** 6, -1])                   # n > L, past its table, negative
    status.zero_()
    pa.pa_decode_tree(b.out, b.q, b.k, b.v, i32(b.p.tables), lens, i32(b.starts), b.scale,
                      tree_mask=i32(b.mask), max_q_len=7, max_seq_len=2 * 10 ** 6, status=status)
    assert int(status) == 5
    b.check(skip=(0, 2, 3))


def test_bad_blocks_read_zeros(pa):
    b = Batch([40, 100], [4, 5], 8, 2, 128, 16, "bf16")
    b.p.tables[1, 2] = b.p.NB + 5
    b.p.tables[0, 0] = -3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.run(pa, status=status)
    assert int(status) == 5
    k, v = b.k.clone(), b.v.clone()
    for pool in (k, v):                                # a spare block of zeros in their place
        pool[b.p.NB - 1] = pool[b.p.NB - 1]
    spare = [i for i in range(b.p.NB) if i not in b.p.tables]
    k[spare[0]] = 0
    v[spare[0]] = 0
    b.k, b.v = k, v
    b.p.tables[1, 2] = b.p.tables[0, 0] = spare[0]
    b.check()


def test_rows_behind_the_last_sequence_stay(pa):
    b = Batch([40, 100], [4, 5], 8, 2, 128, 16, "bf16")
    out = torch.full((12, 8, 128), 7.0, dtype=b.dt, device="cuda")
    q = torch.cat([b.q, b.q[:3]])
    mask = np.concatenate([b.mask, b.mask[:3]])
    pa.pa_decode_tree(out, q, b.k, b.v, i32(b.p.tables), i32(b.lens), i32(b.starts), b.scale,
                      tree_mask=i32(mask), max_q_len=5)
    assert (out[9:] == 7.0).all()
    b.out = out[:9]
    b.check()


def test_offsets_past_32_bits(pa):
    """A pool of more than 2^31 elements: rows of its last blocks."""
    H, D, bs = 8, 128, 64
    NB = (1 << 31) // (H * D * bs) + 40
    k = torch.zeros(NB, bs, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    b = Batch([600], [5], 16, H, D, bs, "bf16")
    used = -(-600 // bs)
    tables = np.arange(NB - used, NB, dtype=np.int32)[None]
    k[NB - used:] = b.k[torch.from_numpy(b.p.tables[0, :used].astype(np.int64)).cuda()]
    v[NB - used:] = b.v[torch.from_numpy(b.p.tables[0, :used].astype(np.int64)).cuda()]
    pa.pa_decode_tree(b.out, b.q, k, v, i32(tables), i32(b.lens), i32(b.starts), b.scale,
                      tree_mask=i32(b.mask), max_q_len=5)
    b.check()


def test_a_bound_whose_costs_pass_32_bits(pa):
    """max_seq_len may be far more than the lengths are: the shares are then counted in 64 bits."""
    g = np.random.default_rng(8)
    lens = [int(x) for x in g.integers(1, 900, size=70)]
    counts = [int(min(n, x)) for n, x in zip(lens, g.integers(0, 9, size=70))]
    b = Batch(lens, counts, 16, 8, 128, 16, "bf16")
    assert 70 * 8 * 4 * ((1 << 30) // 128) > 1 << 31
    b.run(pa, max_seq_len=(1 << 30) - 1).check()


@pytest.mark.parametrize("Hq,H", [(96, 1), (130, 2), (70, 1), (12, 4)])
def test_heads_that_do_not_fill_a_group(pa, Hq, H):
    """More query heads to a KV head than columns of a product, and odd shares of them."""
    Batch([200, 7, 300], [3, 1, 2], Hq, H, 64, 16, "bf16").run(pa).check()


def test_the_tree_mask_helper(pa):
    g = np.random.default_rng(3)
    parents = [chain_or_tree(n, "tree", g) for n in (5, 40, 1)]
    got = pa.tree_mask(parents).cpu().numpy()
    assert np.array_equal(got, np.concatenate([words_of(p, 2) for p in parents]))
    with pytest.raises(ValueError):
        pa.tree_mask([[0]])


def test_graphs_that_share_a_workspace(pa):
    """Two captured calls on one stream with one workspace, replayed on new inputs."""
    a, b = (Batch([3000, 900], [4, 30], 8, 2, 128, 16, "bf16", seed=s) for s in (1, 2))
    ws = pa.workspace_for_tree(a.q, a.k, 30)
    keep = [(x.args(), i32(x.mask)) for x in (a, b)]

    def step():
        for args, mask in keep:
            pa.pa_decode_tree(*args, tree_mask=mask, max_q_len=30, max_seq_len=3000, workspace=ws)
    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    a.q.copy_(a.q.flip(0))
    b.q.neg_()
    for x in (a, b):
        x.out.fill_(7.0)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()
    first = a.out.clone()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, a.out)                     # the same bits every time


def test_two_streams_at_once(pa):
    xs = [Batch([5000, 70], [4, 30], 8, 2, 128, 16, "bf16", seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in xs]
    kw = [dict(tree_mask=i32(x.mask), max_q_len=30, max_seq_len=5000) for x in xs]
    args = [x.args() for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ar, k in zip(streams, args, kw):
            pa.pa_decode_tree(*ar, stream=s, **k)
    torch.cuda.synchronize()
    for x in xs:
        x.check()

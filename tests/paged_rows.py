"""What the tests of the drafted trees and the latent cache share: batches over a paged pool,
and the bound of an attention output.

Bound.  u = 2^-24.  A score is a sum of Dk exact products in fp32, off by at most Dk u of
the sum of magnitudes, twice that where the tensor cores truncate.  A weight is off by that
(times ln 2 of the base-2 form, and times log2 e again), by 2^-20 for the power of two, its
argument and the running maximum, and by its rounding before the product with V: half a
step of the storage type, or 2^-14 of two terms.  The sums over the tokens are fp32 too: an
error of (tokens) u of sum w |v| in the worst order, taken for 4,096 of them as 2^-12.  The
weights' sum is off alike, so the quotient by twice that; and the store by half a step."""
import numpy as np
import torch

from oracle import latent as ol

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.detach().double().cpu().numpy()


def bound(ref, mag, size, Dk, dt, terms):
    """Largest error of an output [n, Dv] by its magnitudes."""
    half = torch.finfo(dt).eps / 2
    tiny = float(torch.finfo(dt).smallest_normal) * half
    score = 2 * Dk * 2.0 ** -24 * size[:, None]
    weight = score + 2.0 ** -20 + (half if terms == 1 else 2.0 ** -14) + 2.0 ** -12
    err = 2 * weight * mag
    return half * (np.abs(ref) + err) + err + tiny


def assert_rows(got, ref, mag, size, Dk, dt, terms, what=""):
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)), (what, int((fine != np.isfinite(got)).sum()))
    b = bound(ref, mag, size, Dk, dt, terms)
    with np.errstate(invalid="ignore"):
        bad = fine & (np.abs(got - ref) > b)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


def chain_or_tree(n, kind, g):
    """Parents of n drafted tokens."""
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    return [int(g.integers(-1, i)) if i else -1 for i in range(n)]


def words_of(parents, W):
    seen, rows = [], []
    for i, p in enumerate(parents):
        seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        rows.append([(seen[i] >> (32 * w)) & 0xFFFFFFFF for w in range(W)])
    return np.array(rows, dtype=np.uint32).reshape(-1, W).view(np.int32)


class Pages:
    """Sequences of `lens` tokens over a pool with spare blocks, tables in no order; everything
    behind a sequence's end, and every spare block, holds NaN and infinities."""

    def __init__(self, lens, bs, g, spare=3, wide=1):
        self.lens, self.bs = list(lens), bs
        used = [-(-max(0, n) // bs) for n in lens]
        self.NB = sum(used) + spare
        order = g.permutation(self.NB)
        self.tables = np.full((len(lens), max(used + [0]) + wide), 1 << 30, dtype=np.int32)
        at = 0
        for b, n in enumerate(used):
            self.tables[b, :n] = order[at:at + n]
            at += n
        self.live = np.zeros((self.NB, bs), dtype=bool)
        for b, L in enumerate(lens):
            t = np.arange(max(0, L))
            self.live[self.tables[b, t // bs], t % bs] = True

    def pool(self, row, dt, g, size=1.0):
        """[NB, bs, *row] normal values, and what no token may read."""
        x = torch.from_numpy(g.normal(size=(self.NB, self.bs, *row)) * size).to(dt)
        bad = torch.from_numpy(g.choice([np.nan, np.inf, -np.inf], size=(self.NB, self.bs)))
        live = torch.from_numpy(self.live).reshape(self.NB, self.bs, *[1] * len(row))
        return torch.where(live, x, bad.to(dt).reshape(live.shape)).cuda()

    def rows(self, pool64, b):
        return ol.rows_of(pool64, self.tables[b], self.lens[b], self.bs)


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)

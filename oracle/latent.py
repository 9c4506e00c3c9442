"""fp64 definitions of attention over drafted trees and of the latent cache (numpy).

What a new token sees is a set: every older token of its sequence and the new ones whose
bit its row of the tree mask has set (no mask: itself and the new ones before it)."""
from __future__ import annotations

import numpy as np


def visible(n: int, L: int, words=None) -> np.ndarray:
    """[n, L] bool: what each of a sequence's last n of L tokens sees.  words [n, W] int32."""
    seen = np.ones((n, L), dtype=bool)
    if words is None:
        seen[:, L - n:] = np.tril(np.ones((n, n), dtype=bool))
    else:
        w = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
        for j in range(n):
            seen[:, L - n + j] = (w[:, j // 32] >> (j % 32)) & 1
    return seen


def attend(q, k, v, seen, scale):
    """softmax(scale q k^T) v of one head: q [n, Dk], k [L, Dk], v [L, Dv], seen [n, L].  Also
    the same with |v|, and sum |q k| scale of the largest term of each row: what rounding
    errors are measured by.  A row that sees nothing, or only scores of -inf, is zeros; what a
    row does not see has no part in it, whatever it holds."""
    n, L = seen.shape
    out = np.zeros((n, v.shape[1]))
    mag = np.zeros_like(out)
    size = np.zeros(n)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(n):
            at = np.flatnonzero(seen[i])
            if at.size == 0:
                continue
            s = scale * (k[at] @ q[i])
            size[i] = abs(scale) * (np.abs(k[at]) @ np.abs(q[i])).max()
            top = s.max()
            if top == -np.inf:
                continue
            p = np.exp(s - top)
            out[i] = (p @ v[at]) / p.sum()
            mag[i] = (p @ np.abs(v[at])) / p.sum()
    return out, mag, size


def rows_of(pool, table, n, block_size):
    """The first n rows of a sequence: pool [NB, bs, ...], its blocks in table order."""
    t = np.arange(n)
    return pool[np.asarray(table)[t // block_size], t % block_size]

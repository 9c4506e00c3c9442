"""fp64 norm + rotation of new tokens, and the 8-bit cache (oracle side).

Rotation: a head row x at position p, with the row (c_0 .. c_{R/2-1}, s_0 ..) of the
cos_sin table, maps each pair (a, b) to (x_a c - x_b s, x_b c + x_a s); pairs are
(j, j + R/2), or (2j, 2j + 1) when interleaved.  RMS norm: x / sqrt(mean(x^2) + eps) * w.

The cache holds e4m3 codes and one scale per (block, KV head); a stored value is
code * scale.  e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits, subnormals, no
infinities, NaN = 0x7F / 0xFF, largest value 448.
"""
from __future__ import annotations

import math

import numpy as np

MIN_EXP = -64


def _positive_values() -> np.ndarray:
    """Values of the codes 0x00 .. 0x7E, ascending."""
    out = []
    for code in range(0x7F):
        e, f = code >> 3, code & 7
        out.append(f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(out)


VALUES = _positive_values()


def decode_e4m3(codes: np.ndarray) -> np.ndarray:
    codes = np.asarray(codes, dtype=np.uint8)
    low = codes & 0x7F
    v = np.where(low == 0x7F, np.nan, VALUES[np.minimum(low, 0x7E)])
    return np.where(codes & 0x80, -v, v)


def encode_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even code; beyond 448 (infinities too) the largest;
    NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    mid = (VALUES[:-1] + VALUES[1:]) / 2
    lo = np.searchsorted(mid, a, side="left")           # mid[lo - 1] < a <= mid[lo]
    tie = (lo < len(mid)) & (a == mid[np.minimum(lo, len(mid) - 1)])
    code = np.where(tie & (lo & 1 == 1), lo + 1, lo).astype(np.uint8)
    code = np.where(np.isnan(x), 0x7F, code).astype(np.uint8)
    return np.where(np.signbit(x) & ~np.isnan(x), code | 0x80, code).astype(np.uint8)


def scale_for(amax: float) -> float:
    """The smallest 2^e, e >= MIN_EXP, with amax <= 448 * 2^e."""
    if amax == 0:
        return 2.0 ** MIN_EXP
    m, x = math.frexp(amax / 448.0)                     # amax / 448 = m 2^x, m in [1/2, 1)
    return 2.0 ** max(MIN_EXP, x - 1 if m == 0.5 else x)


def finite_amax(x: np.ndarray) -> float:
    a = np.abs(x)
    a = a[np.isfinite(a)]
    return float(a.max()) if a.size else 0.0


def rms_norm(x: np.ndarray, weight, eps: float) -> np.ndarray:
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotate(x: np.ndarray, angles: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [..., heads, D]; angles [..., R] (cosines, then sines)."""
    R = angles.shape[-1]
    y = x.copy()
    for j in range(R // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        c, s = angles[..., None, j], angles[..., None, R // 2 + j]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def placements(seq_lens, q_start, block_tables, block_size):
    """(token row, sequence, position, block, row) of every new token."""
    out = []
    for b, L in enumerate(seq_lens):
        s, e = (b, b + (1 if L else 0)) if q_start is None else (q_start[b], q_start[b + 1])
        for t in range(s, e):
            pos = int(L) - (e - s) + t - s
            out.append((t, b, pos, int(block_tables[b][pos // block_size]), pos % block_size))
    return out


def append_q8(codes: np.ndarray, scales: np.ndarray, rows: np.ndarray, places) -> None:
    """New rows ([T, H, D] float64) into codes [NB, H, bs, D] / scales [NB, H], in place."""
    by_block = {}
    for t, _, _, block, row in places:
        by_block.setdefault(block, []).append((row, t))
    for block, items in by_block.items():
        items.sort()
        first = items[0][0]
        for h in range(codes.shape[1]):
            new = np.stack([rows[t, h] for _, t in items])
            s = scale_for(finite_amax(new))
            if first > 0:
                old = float(scales[block, h])
                if s > old:
                    kept = decode_e4m3(codes[block, h, :first])
                    codes[block, h, :first] = encode_e4m3(kept * (old / s))
                s = max(s, old)
            for row, t in items:
                codes[block, h, row] = encode_e4m3(rows[t, h] / s)
            scales[block, h] = s


def values_q8(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 pool [NB, bs, H, D] of an 8-bit cache."""
    v = decode_e4m3(codes) * np.asarray(scales, dtype=np.float64)[:, :, None, None]
    return v.transpose(0, 2, 1, 3)


def decode_with_spread(q, k_pool, v_pool, table, length, scale):
    """One sequence: (out, sum_t p_t |V_t|, max_t scale sum_d |q_d K_td|), each per query
    head, from float64 pools [NB, bs, H, D]; the last two enter error bounds."""
    Hq, D = q.shape
    bs, H = k_pool.shape[1], k_pool.shape[2]
    G = Hq // H
    if length == 0:
        return np.zeros((Hq, D)), np.zeros((Hq, D)), np.zeros(Hq)
    pos = np.arange(length)
    blk = np.asarray(table, dtype=np.int64)[pos // bs]
    out, mass, size = np.empty((Hq, D)), np.empty((Hq, D)), np.empty(Hq)
    for h in range(H):
        k, v = k_pool[blk, pos % bs, h], v_pool[blk, pos % bs, h]
        for g in range(h * G, (h + 1) * G):
            s = scale * (k @ q[g])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[g], mass[g] = p @ v, p @ np.abs(v)
            size[g] = scale * (np.abs(k) @ np.abs(q[g])).max()
    return out, mass, size

"""How exact the 8-bit cache's decode attention is where its digits could lose something:
weights of any size, blocks of one sequence whose V scales are far apart, a q with one
large channel, against the definition in fp64.

Bounds, for one query head, with p the softmax weights, w_t = p_t (V scale of t's block),
A = sum_t p_t |V_t| and C = sum_t |code of V_t| per output element, U = max_t w_t, and
S = max_t scale sum_d |q_d K_td|:
  - scores: at most 3 x 128 products summed in fp32, 384 * 2^-24 S = 2^-15.4 S in natural
    units; with a score off by x, weight and normaliser are off by a factor of e^(2x);
  - weights: three e4m3 digits of an fp32 number, 2^-14 of each (four bits of it, then five
    and five of what is left), of which the last two may go by fp16, whose half step is
    2^-12 of at most 2^-4 of it: 2^-13.6 in all;
  - q: its digits' last steps are 2^-17 where the row's largest |q| is between 224 and 448,
    so an element is exact where its own last bit is 2^-17 or more, and off by 2^-18 / 224 =
    2^-25.8 of the largest otherwise (only where a test has such elements);
  - the last digit's steps are 2^-17 where the tile's largest w is between 128 and 256, so
    half a step is at most 2^-25 U of a w, and that many codes: 2^-25 U C;
  - exponentials, products and sums in fp32: taken as 2^-16 A;
  - the store: half a step of the type."""
import numpy as np
import pytest
import torch

from oracle import cache_q8 as oq
from tests.gpu_helpers import lib
from tests.test_gpu_cache_q8 import Batch, f64

pytestmark = pytest.mark.gpu
WEIGHT = 2.0 ** -13.6


@pytest.fixture(scope="module")
def pa():
    return lib()


def check(b, out, inexact_q=False):
    """`out` against fp64 attention over b's codes and scales, within the bounds above."""
    half = torch.finfo(b.dt).eps / 2
    tiny = float(torch.finfo(b.dt).smallest_normal) * half
    q, got = f64(b.q), f64(out)
    values = [oq.values_q8(c, s) for c, s in zip(b.codes, b.scales)]
    for i, n in enumerate(b.lens):
        if n == 0:
            continue
        pos = np.arange(n)
        blk = b.tables[i, pos // b.bs]
        for hq in range(q.shape[1]):
            h = hq * b.H // q.shape[1]
            k, v = (x[blk, pos % b.bs, h] for x in values)
            s = b.scale * (k @ q[i, hq])
            p = np.exp(s - s.max())
            p /= p.sum()
            size = b.scale * (np.abs(k) @ np.abs(q[i, hq])).max()
            scale_v = b.scales[1][blk, h].astype(np.float64)
            a = p @ np.abs(v)
            c = (np.abs(v) / scale_v[:, None]).sum(0)
            off = 2.0 ** -15.4 * size                     # of a score
            if inexact_q:
                off += b.scale * 2.0 ** -25.8 * np.abs(q[i, hq]).max() * np.abs(k).sum(1).max()
            e = (WEIGHT + np.expm1(2 * off) + 2.0 ** -16) * a + 2.0 ** -25 * (p * scale_v).max() * c
            ref = p @ v
            bad = ~(np.abs(got[i, hq] - ref) <= half * (np.abs(ref) + e) + e + tiny)
            assert not bad.any(), (i, hq, int(bad.sum()), np.abs(got[i, hq] - ref).max(), ref[bad][:3])


def put(b):
    """b's codes and scales to the GPU."""
    for x, y in zip(b.pools + b.sc, b.codes + b.scales):
        x.copy_(torch.from_numpy(y))


def lean(b, i, blocks, by):
    """Sequence i's scores in `blocks` (places in its table) rise by `by` (base 2) over what
    they are elsewhere, by K's first channel; its second one spreads them by a factor of a
    few, and q sees no other."""
    b.q[i] = 0
    b.q[i, :, 0] = 1
    b.q[i, :, 1] = 1.0 / by
    for j in range(-(-b.lens[i] // b.bs)):
        blk = b.tables[i, j]
        n = min(b.bs, b.lens[i] - j * b.bs)
        b.codes[0][blk, :, :n, 0] = oq.encode_e4m3(np.array(64.0 if j in blocks else 0.0))
        b.scales[0][blk] = by * np.log(2.0) / b.scale / 64.0


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 2), (128, 5), (128, 8), (64, 4), (64, 7)])
def test_weights_keep_their_bits(pa, D, G, dt):
    """Three tokens: the first has the largest weight and no V, the others opposite V, so
    that the output is the difference of their weights."""
    b = Batch([3] * 40, G, 2, D, 16, dt, seed=G)
    g = np.random.default_rng(D + G)
    b.q.zero_()
    b.q[:, :, 0] = torch.from_numpy(g.uniform(0.5, 1, size=b.q.shape[:2])).to(b.dt)
    for i in range(len(b.lens)):
        blk = b.tables[i, 0]
        b.codes[0][blk, :, 0, 0] = oq.encode_e4m3(np.array(64.0))
        b.codes[0][blk, :, 1:3, 0] = oq.encode_e4m3(g.uniform(-60, 60, size=(2, 2)))
        b.scales[0][blk] = 1.0 / (64 * b.scale)              # scores of 1 and less
        b.codes[1][blk, :, 0] = 0
        b.codes[1][blk, :, 2] = b.codes[1][blk, :, 1] ^ 0x80
    put(b)
    check(b, b.run(pa))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (128, 5), (128, 8), (64, 2), (64, 8)])
@pytest.mark.parametrize("apart", [16, 20, 24, 30, 60])
def test_a_block_of_large_scale_and_no_weight(pa, D, G, dt, apart):
    """A tile of eight blocks: one has a V scale 2^apart times the others' and 2^-(apart + 6)
    of their weight.  The others decide the output, and keep their bits."""
    b = Batch([128, 100, 1000], G, 2, D, 16, dt, seed=apart)
    for i, n in enumerate(b.lens):
        used = -(-n // 16)
        lean(b, i, [j for j in range(used) if j != 2], apart + 6)
        for j in range(used):
            b.scales[1][b.tables[i, j]] = 2.0 ** (apart - 6 if j == 2 else -6)
    put(b)
    check(b, b.run(pa))


@pytest.mark.parametrize("D,G", [(128, 3), (64, 4)])
def test_scales_over_their_whole_range(pa, D, G):
    """V scales from 2^-100 to 2^80, block by block, with weights that make up for them or
    do not: every sequence's own largest weight times scale sets its bits."""
    spans = [(-40, 81), (-100, 81), (-64, 20), (-100, -60), (-64, 64)]
    b = Batch([64, 128, 200, 777, 1300], G, 2, D, 8, "bf16", seed=3)
    g = np.random.default_rng(5)
    for i, (n, span) in enumerate(zip(b.lens, spans)):
        used = -(-n // 8)
        b.scales[1][b.tables[i, :used]] = 2.0 ** g.integers(*span, size=(used, 2))
    put(b)
    check(b, b.run(pa))


@pytest.mark.parametrize("D,G", [(128, 4), (64, 5)])
@pytest.mark.parametrize("by", [100, 140, 400])
def test_a_tile_far_below_the_running_maximum(pa, D, G, by):
    """Later tiles whose weights are 2^-by of the first one's: they add next to nothing, or
    nothing, and no NaN; and first ones that a later tile leaves that far behind."""
    b = Batch([512, 700, 640], G, 2, D, 16, "bf16", seed=by)
    lean(b, 0, range(0, 8), by)
    lean(b, 1, range(40, 44), by)
    lean(b, 2, [], by)                       # weights of one size throughout
    for i in (0, 1):
        used = -(-b.lens[i] // 16)
        b.scales[1][b.tables[i, :used]] = 2.0 ** -70
        b.scales[1][b.tables[i, 20]] = 2.0 ** 30
    put(b)
    out = b.run(pa)
    assert torch.isfinite(out).all()
    check(b, out)


@pytest.mark.parametrize("dt,large,exact", [("bf16", 2 ** 7, True), ("bf16", 2 ** 16, True),
                                            ("bf16", 2 ** 20, False), ("bf16", 2 ** 24, False),
                                            ("fp16", 2 ** 7, True), ("fp16", 2 ** 13, True),
                                            ("fp16", 2 ** 15, False)])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (64, 8)])
def test_one_large_channel_of_q(pa, D, G, dt, large, exact):
    """One channel of q is large and K is zero there: the others, from 1/2 to 2 in size, decide
    the scores."""
    b = Batch([1, 100, 300], G, 2, D, 16, dt, seed=D + G)
    g = np.random.default_rng(G)
    q = g.uniform(0.5, 2, size=b.q.shape) * g.choice([-1, 1], size=b.q.shape)
    q[..., 7] = large
    b.q.copy_(torch.from_numpy(q))
    for i, n in enumerate(b.lens):
        blk = b.tables[i, :-(-n // 16)]
        b.codes[0][blk, :, :, 7] = 0
        b.scales[0][blk] = 2.0 ** -8
    put(b)
    check(b, b.run(pa), inexact_q=not exact)

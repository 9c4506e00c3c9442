"""GPU parity of the rotated cache writes (16-bit and 8-bit) against the fp64 oracle.

Bounds.  u = 2^-24.  The norm's factor: 13 roundings in the sum of squares (8 in a lane,
then 4 halving steps), halved by the root, the division, the addition of eps and a
rsqrt of 2 ulp (4 u): at most 13 u; then two products (2 u) and the rotation (two
products and a difference: 2 u): 17 u of |x_a| + |x_b|, taken as 20 u.  The store adds half
a step of the storage type, eps / 2 of the value (bf16 2^-8, fp16 2^-11), or half a
subnormal step.  A code is off by at most half a step: 2^-4 of its value or 2^-10, in
units of the scale, on top of the fp32 error.  Values are exact: 16-bit copies, and codes
of exact quotients by a power of two."""
import numpy as np
import pytest
import torch

from oracle import cache_q8 as oq
from tests.gpu_helpers import i32, lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def pa():
    return lib()


def f64(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """Random tokens, tables and pools; `new` None: a decode step."""

    def __init__(self, lens, new, Hq, H, D, bs, dt, R, interleaved=False, norm="", packed=False,
                 positions=False, behind=0, seed=0):
        g = np.random.default_rng(seed + 1000 * D + bs)
        self.lens, self.new, self.Hq, self.H, self.D, self.bs = lens, new, Hq, H, D, bs
        self.R, self.interleaved, self.dt = R, interleaved, DT[dt]
        B = len(lens)
        used = [-(-n // bs) for n in lens]
        self.NB = sum(used) + 5
        order = g.permutation(self.NB)
        MB = max(used) + 1
        self.tables = np.full((B, MB), 1 << 30, dtype=np.int32)    # never read past the end
        at = 0
        for b, n in enumerate(used):
            self.tables[b, :n] = order[at:at + n]
            at += n
        self.q_start = None if new is None else np.concatenate([[0], np.cumsum(new)])
        self.T = B if new is None else int(self.q_start[-1]) + behind
        w = (Hq + 2 * H) * D
        x = torch.from_numpy(g.normal(size=(self.T, w + (24 if packed else 0)))
                             * np.exp(g.normal(size=(self.T, 1)))).to(self.dt).cuda()

        def part(lo, heads):
            return x[:, lo:lo + heads * D].unflatten(1, (heads, D))
        self.q, self.k, self.v = part(0, Hq), part(Hq * D, H), part((Hq + H) * D, H)
        if not packed:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))

        def weight(on):
            return torch.from_numpy(g.uniform(0.5, 1.5, D)).to(self.dt).cuda() if on else None
        self.qw, self.kw = weight("q" in norm), weight("k" in norm)
        P = max(lens) + 7
        th = g.uniform(-np.pi, np.pi, size=(P, R // 2))
        self.cs = torch.from_numpy(np.concatenate([np.cos(th), np.sin(th)], 1)).float().cuda() \
            if R else None
        self.pos = i32(g.integers(0, P, size=self.T)) if positions else None
        self.places = oq.placements(lens, self.q_start, self.tables, bs)
        self.q_out = torch.from_numpy(g.normal(size=(self.T, Hq, D))).to(self.dt).cuda()
        self.q_before = f64(self.q_out)
        self.g = g

    def kw_args(self):
        return dict(q_start=None if self.q_start is None else i32(self.q_start), q_weight=self.qw,
                    k_weight=self.kw, eps=1e-5, interleaved=self.interleaved,
                    positions=self.pos)

    def reference(self, x, w):
        """(fp64 rows, bound of the fp32 error) of every token's heads."""
        y = oq.rms_norm(f64(x), None if w is None else f64(w), 1e-5)
        if not self.R:
            return y, 20 * U * np.abs(y)
        pos = np.zeros(self.T, dtype=np.int64)
        for t, _, p, _, _ in self.places:
            pos[t] = p
        if self.pos is not None:
            pos = self.pos.cpu().numpy()
        cs = f64(self.cs)[pos]
        pair = np.abs(y).copy()
        R = self.R
        a, b = (slice(0, R, 2), slice(1, R, 2)) if self.interleaved else \
            (slice(0, R // 2), slice(R // 2, R))
        pair[..., a] = pair[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
        return oq.rotate(y, cs, self.interleaved), 20 * U * pair

    def close16(self, got, ref, err):
        half = torch.finfo(self.dt).eps / 2
        tiny = float(torch.finfo(self.dt).smallest_normal) * half
        bad = np.abs(got - ref) > half * (np.abs(ref) + err) + err + tiny
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])

    def check_q(self):
        ref, err = self.reference(self.q, self.qw)
        got = f64(self.q_out)
        rows = np.array([p[0] for p in self.places], dtype=np.int64)
        self.close16(got[rows], ref[rows], err[rows])
        rest = np.setdiff1d(np.arange(self.T), rows)
        assert np.array_equal(got[rest], self.q_before[rest])      # left as they were


STEP = [1, 16, 17, 33, 64, 5, 0, 40]
RAGGED = ([40, 7, 64, 130, 9, 1, 65], [40, 3, 0, 100, 9, 1, 2])
MANY = ([1 + (7 * i) % 50 for i in range(100)], [min(1 + (7 * i) % 50, (i * i) % 5) for i in range(100)])

CASES = [
    # lens, new, Hq, H, D, bs, dt, R, further
    (STEP, None, 4, 4, 64, 16, "fp16", 64, dict(interleaved=True)),
    (STEP, None, 32, 8, 128, 16, "bf16", 128, dict(norm="qk", packed=True)),
    (STEP, None, 5, 1, 128, 32, "fp16", 64, dict(norm="k")),
    (STEP, None, 7, 7, 64, 8, "bf16", 16, dict(norm="q", packed=True)),
    (STEP, None, 3, 3, 128, 64, "bf16", 0, dict(norm="qk")),
    (STEP, None, 12, 3, 64, 64, "fp16", 48, dict(positions=True)),
    (*RAGGED, 8, 2, 128, 16, "bf16", 128, dict(norm="qk")),
    (*RAGGED, 6, 3, 64, 8, "fp16", 32, dict(interleaved=True, packed=True, behind=5)),
    (*RAGGED, 4, 1, 128, 64, "fp16", 112, dict(norm="k", positions=True)),
    (*RAGGED, 40, 8, 128, 32, "bf16", 64, dict(packed=True, behind=3)),
    (*RAGGED, 2, 2, 64, 16, "bf16", 64, dict(norm="qk", interleaved=True)),
    (*RAGGED, 9, 3, 64, 32, "fp16", 16, dict()),
    (*RAGGED, 16, 2, 128, 8, "fp16", 0, dict()),
    (*RAGGED, 2, 1, 64, 64, "bf16", 64, dict(norm="qk")),
    (*MANY, 4, 2, 128, 16, "bf16", 128, dict(norm="qk")),
    (*MANY, 4, 2, 64, 8, "fp16", 64, dict(behind=9)),
    ([300], [300], 3, 1, 128, 16, "bf16", 128, dict(norm="q", interleaved=True)),
    ([70] + [2] * 66, [70] + [1] * 66, 4, 4, 64, 64, "fp16", 64, dict(norm="k")),
    # enough tokens for the ring of shared-memory stages (8 per SM), with other shapes of it
    ([1500, 3, 900, 1], [1400, 0, 900, 1], 4, 2, 128, 16, "bf16", 128, dict(norm="qk", packed=True)),
    ([1500, 3, 900, 1], [1400, 2, 900, 1], 6, 3, 64, 8, "fp16", 32,
     dict(interleaved=True, behind=5, positions=True)),
    ([2500], [2400], 96, 1, 128, 64, "fp16", 64, dict(norm="q")),
    ([2500], [2400], 1, 1, 64, 32, "bf16", 0, dict(norm="k")),
    # a ring whose stages take just under 48 KB
    ([2500], [2400], 14, 2, 64, 16, "bf16", 16, dict(norm="qk")),
    ([1 + (7 * i) % 40 for i in range(1300)], [min(1 + (7 * i) % 40, 1 + i % 2) for i in range(1300)],
     2, 2, 128, 16, "bf16", 128, dict(norm="k")),
]


def _setup(case, seed):
    lens, new, Hq, H, D, bs, dt, R, more = case
    return Setup(lens, new, Hq, H, D, bs, dt, R, seed=seed, **more)


@pytest.mark.parametrize("n", range(len(CASES)))
def test_rope_append(pa, n):
    s = _setup(CASES[n], n)
    kp = torch.from_numpy(s.g.normal(size=(s.NB, s.bs, s.H, s.D))).to(s.dt).cuda()
    vp = torch.from_numpy(s.g.normal(size=(s.NB, s.bs, s.H, s.D))).to(s.dt).cuda()
    want_k, want_v = f64(kp), f64(vp)
    before_k = want_k.copy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.pa_rope_append(s.q_out, kp, vp, s.q, s.k, s.v, s.cs, i32(s.tables), i32(s.lens),
                            status=status, **s.kw_args())
    torch.cuda.synchronize()
    assert out is s.q_out and int(status.item()) == 0
    s.check_q()
    ref, err = s.reference(s.k, s.kw)
    got = f64(kp)
    v = f64(s.v)
    for t, _, _, block, row in s.places:
        s.close16(got[block, row], ref[t], err[t])
        got[block, row] = before_k[block, row]
        want_v[block, row] = v[t]
    assert np.array_equal(got, before_k)            # no other row changed
    assert np.array_equal(f64(vp), want_v)


def _cache(s):
    """Codes without NaN where sequences live, NaN codes elsewhere; scales near those of
    the new rows, so that some blocks grow and some do not."""
    codes = [s.g.integers(0, 0x7F, size=(s.NB, s.H, s.bs, s.D)).astype(np.uint8)
             | (s.g.integers(0, 2, size=(s.NB, s.H, s.bs, s.D)) * 0x80).astype(np.uint8)
             for _ in range(2)]
    for c in codes:
        live = np.zeros((s.NB, s.bs), dtype=bool)
        for b, L in enumerate(s.lens):
            pos = np.arange(L)
            live[s.tables[b, pos // s.bs], pos % s.bs] = True
        c.transpose(0, 2, 1, 3)[~live] = 0x7F
    scales = [(2.0 ** s.g.integers(-12, -3, size=(s.NB, s.H))).astype(np.float32)
              for _ in range(2)]
    return codes, scales


@pytest.mark.parametrize("n", range(len(CASES)))
def test_rope_append_q8(pa, n):
    s = _setup(CASES[n], n + 100)
    codes, scales = _cache(s)
    pools = [torch.from_numpy(c.copy()).cuda() for c in codes]
    sc = [torch.from_numpy(x.copy()).cuda() for x in scales]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_rope_append_q8(s.q_out, pools[0], pools[1].view(pa.E4M3), sc[0], sc[1], s.q, s.k, s.v,
                         s.cs, i32(s.tables), i32(s.lens), status=status, **s.kw_args())
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    s.check_q()
    ref, err = s.reference(s.k, s.kw)
    for i, rows in enumerate((ref, f64(s.v))):
        want_c, want_s = codes[i].copy(), scales[i].astype(np.float64)
        oq.append_q8(want_c, want_s, rows, s.places)
        got_c, got_s = pools[i].cpu().numpy(), f64(sc[i])
        assert np.array_equal(got_s, want_s)
        if i == 0:           # the new keys: half a code step and the fp32 error
            for t, _, _, block, row in s.places:
                x = ref[t] / want_s[block][:, None]
                e = err[t] / want_s[block][:, None]
                d = np.abs(oq.decode_e4m3(got_c[block, :, row]) - x)
                assert (d <= np.maximum(2.0 ** -4 * (np.abs(x) + e), 2.0 ** -10) + e).all()
                got_c[block, :, row] = want_c[block, :, row]
        assert np.array_equal(got_c, want_c)        # everything else to the bit


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_in_place(pa, dt):
    """q_out = q, packed."""
    s = Setup(*RAGGED, 8, 2, 128, 16, dt, 128, norm="qk")
    kp = torch.zeros(s.NB, s.bs, s.H, s.D, dtype=s.dt, device="cuda")
    vp = torch.zeros_like(kp)
    args = (s.k, s.v, s.cs, i32(s.tables), i32(s.lens))
    pa.pa_rope_append(s.q_out, kp, vp, s.q, *args, **s.kw_args())
    q2 = s.q.clone()
    pa.pa_rope_append(q2, kp, vp, q2, *args, **s.kw_args())
    torch.cuda.synchronize()
    assert torch.equal(q2, s.q_out)


def test_many_tokens_in_place_and_past_a_bad_one(pa):
    """The ring's writes over its own reads; a token outside the table and a bad block in
    the middle of a run are left alone."""
    s = Setup([2000, 700], [2000, 700], 8, 2, 128, 16, "bf16", 128, norm="qk")
    pos = np.array([p[2] for p in s.places])
    pos[1234] = s.cs.shape[0]
    tables = s.tables.copy()
    tables[1, 3] = -5
    kw = s.kw_args() | dict(positions=i32(pos))
    kp = torch.full((s.NB, s.bs, s.H, s.D), 9.0, dtype=s.dt, device="cuda")
    vp = kp.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = f64(s.q)[1234]
    q2 = s.q.clone()
    pa.pa_rope_append(q2, kp, vp, q2, s.k, s.v, s.cs, i32(tables), i32(s.lens), status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 5
    got = f64(q2)
    assert np.array_equal(got[1234], before)
    ref, err = s.reference(s.q, s.qw)
    rows = np.array([t for t in range(s.T) if t != 1234])
    s.close16(got[rows], ref[rows], err[rows])
    v, stored = f64(s.v), f64(vp)
    for t, b, p, block, row in s.places:
        left = t == 1234 or (b == 1 and p // 16 == 3)
        assert np.array_equal(stored[block, row], np.full_like(v[t], 9.0) if left else v[t])


def test_step_form_and_general_form_agree(pa):
    """q_start None and one token per sequence given by q_start: the same bits."""
    lens = [n for n in STEP if n]
    s = Setup(lens, None, 8, 4, 128, 16, "bf16", 128, norm="qk")
    codes, scales = _cache(s)
    got = []
    for start in (None, i32(np.arange(len(lens) + 1))):
        pools = [torch.from_numpy(c.copy()).cuda() for c in codes]
        sc = [torch.from_numpy(x.copy()).cuda() for x in scales]
        kw = s.kw_args() | dict(q_start=start)
        q = torch.empty_like(s.q)
        pa.pa_rope_append_q8(q, *pools, *sc, s.q, s.k, s.v, s.cs, i32(s.tables), i32(lens), **kw)
        torch.cuda.synchronize()
        got.append([q.view(torch.int16), *pools, *sc])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("step", [True, False])
def test_infinities_and_nan(pa, step):
    """An infinity becomes the largest code and a NaN a NaN code; neither sets the scale."""
    s = Setup([20], None if step else [4], 1, 1, 64, 16, "fp16", 0)
    s.k[-1, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 7.0])
    s.k[-1, 0, 4:] = 0.5
    s.v[-1].fill_(float("nan"))
    if not step:
        s.k[:-1].fill_(0.25)
        s.v[:-1].zero_()
    codes = [torch.zeros(s.NB, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.full((s.NB, 1), 2.0 ** -20, device="cuda") for _ in range(2)]
    pa.pa_rope_append_q8(s.q_out, *codes, *sc, s.q, s.k, s.v, None, i32(s.tables), i32(s.lens),
                         **s.kw_args())
    torch.cuda.synchronize()
    blk = int(s.tables[0, 1])
    assert float(sc[0][blk, 0]) == 2.0 ** -6                # 7 = 448 * 2^-6
    assert codes[0][blk, 0, 3, :5].tolist() == [0x7E, 0xFE, 0x7F, 0x7E, 0x60]   # 0.5 = 32 * 2^-6
    assert (codes[1][blk, 0, 3] == 0x7F).all()
    # row 3 keeps the older rows' scale; a block written from row 0 has no finite magnitude but 0
    assert float(sc[1][blk, 0]) == (2.0 ** -20 if step else 2.0 ** -64)


def test_zeros_have_the_smallest_scale(pa):
    s = Setup([3], [3], 1, 2, 128, 8, "bf16", 0)
    s.v.zero_()
    codes = [torch.full((s.NB, 2, 8, 128), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.ones(s.NB, 2, device="cuda") for _ in range(2)]
    pa.pa_rope_append_q8(s.q_out, *codes, *sc, s.q, s.k, s.v, None, i32(s.tables), i32(s.lens),
                         **s.kw_args())
    torch.cuda.synchronize()
    blk = int(s.tables[0, 0])
    assert (sc[1][blk] == 2.0 ** -64).all()
    assert not (codes[1][blk, :, :3] & 0x7F).any() and (codes[1][blk, :, 3:] == 7).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("many", [False, True])
def test_bad_row_ranges_are_reported_and_skipped(pa, q8, many):
    """q_start that is negative, falls, or ends past the rows: none of it is followed."""
    n = 1500 if many else 40
    s = Setup([n, 30, 30], [n, 20, 20], 2, 2, 64, 16, "bf16", 64)
    pools = [torch.zeros(s.NB, 2, 16, 64, dtype=torch.uint8, device="cuda") if q8 else
             torch.zeros(s.NB, 16, 2, 64, dtype=s.dt, device="cuda") for _ in "kv"]
    rest = [torch.ones(s.NB, 2, device="cuda") for _ in "kv"] if q8 else []
    f = pa.pa_rope_append_q8 if q8 else pa.pa_rope_append
    for start in ([-(1 << 31), n, n + 20, n + 40], [0, n, n - 1, n + 40], [0, n, n + 20, n + 41],
                  [0, n, n + 20, (1 << 31) - 1], [5, n, n + 20, n + 40]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = s.kw_args() | dict(q_start=i32(start))
        f(s.q_out, *pools, *rest, s.q, s.k, s.v, s.cs, i32(s.tables), i32(s.lens), status=status,
          **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 5, start


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("step", [True, False])
def test_bad_device_data_is_reported_and_skipped(pa, q8, step):
    """A length past the table, more new tokens than the length, a bad block id and a
    position outside the table: each is reported, and the good sequences are written."""
    lens = [20, 21, 22, 23]
    s = Setup(lens, None if step else [3, 3, 3, 3], 2, 2, 64, 16, "bf16", 64)
    lens2 = list(lens)
    lens2[1] = s.tables.shape[1] * 16 + 1
    tables = s.tables.copy()
    tables[2, 1] = s.NB
    kw = s.kw_args()
    pos = torch.tensor([p[2] for p in s.places], dtype=torch.int32)
    pos[-1] = s.cs.shape[0]                           # the last sequence's last token
    kw["positions"] = pos.cuda()
    if not step:
        lens2[0], s.new = 2, None                     # three new tokens of two
    if q8:
        pools = [torch.full((s.NB, 2, 16, 64), 9, dtype=torch.uint8, device="cuda") for _ in "kv"]
        rest = [torch.ones(s.NB, 2, device="cuda") for _ in "kv"]
        f = pa.pa_rope_append_q8
    else:
        pools = [torch.full((s.NB, 16, 2, 64), 9.0, dtype=s.dt, device="cuda") for _ in "kv"]
        rest, f = [], pa.pa_rope_append
    was = [p.clone() for p in pools]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f(s.q_out, *pools, *rest, s.q, s.k, s.v, s.cs, i32(tables), i32(lens2), status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 5
    changed = set()
    for p, w in zip(pools, was):
        d = (p != w).flatten(2).any(2) if not q8 else (p != w).any(3).any(1)
        changed |= {tuple(x) for x in d.nonzero().tolist()}
    good = set()
    for t, b, p, block, row in s.places:
        if b == 3 and p != lens[3] - 1 or b == 0 and step:
            good.add((block, row))
    assert changed == good
    got = f64(s.q_out)
    touched = {t for t in range(s.T) if not np.array_equal(got[t], s.q_before[t])}
    want = {t for t, b, p, _, _ in s.places
            if b == 2 or b == 3 and p != lens[3] - 1 or b == 0 and step}
    assert touched == want


def test_on_another_stream_and_replayed(pa):
    """Captured on a side stream; replayed with other inputs in the same buffers."""
    s = Setup(STEP, None, 8, 2, 128, 16, "bf16", 128, norm="qk")
    codes, scales = _cache(s)

    def buffers():
        return ([torch.from_numpy(c.copy()).cuda() for c in codes]
                + [torch.from_numpy(x.copy()).cuda() for x in scales])
    tables, lens = i32(s.tables), i32(s.lens)
    kw = s.kw_args()
    one, two = buffers(), buffers()
    q1, q2 = torch.zeros_like(s.q), torch.zeros_like(s.q)
    pa.pa_rope_append_q8(q1, *one, s.q, s.k, s.v, s.cs, tables, lens, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    k_in = torch.zeros_like(s.k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_rope_append_q8(q2, *two, s.q, k_in, s.v, s.cs, tables, lens, **kw)
    k_in.copy_(s.k)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and all(torch.equal(a, b) for a, b in zip(one, two))


def test_offsets_past_32_bits(pa):
    """A 16-bit and an 8-bit pool whose last block lies past 2^32 bytes."""
    H, D, bs = 8, 128, 64
    NB = (1 << 32) // (H * D * bs) + 3
    k = torch.randn(1, H, D, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(1, H, D, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(1, H, D, device="cuda", dtype=torch.bfloat16)
    tables, lens = i32([[NB - 1]]), i32([bs])
    kp = torch.zeros(NB, bs, H, D, device="cuda", dtype=torch.bfloat16)
    vp = torch.zeros_like(kp)
    pa.pa_rope_append(torch.empty_like(q), kp, vp, q, k, v, None, tables, lens)
    k8, v8, ks, vs = pa.alloc_cache_q8(NB, H, bs, D)
    pa.pa_rope_append_q8(torch.empty_like(q), k8, v8, ks, vs, q, k, v, None, tables, lens)
    torch.cuda.synchronize()
    assert torch.equal(kp[-1, -1], k[0]) and torch.equal(vp[-1, -1], v[0])
    assert not kp[:-1].any() and not vp[:-1].any()
    for pool, sc, x in ((k8, ks, k), (v8, vs, v)):
        got = pool[-1, :, -1].float() * sc[-1][:, None]
        d = (got - x[0].float()).abs()
        assert (d <= x[0].float().abs() * 2 ** -4 + sc[-1][:, None] * 2 ** -10).all()
        assert not pool[:-1].view(torch.uint8).any()

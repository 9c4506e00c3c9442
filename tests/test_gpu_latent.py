"""GPU parity of the latent cache's calls against the fp64 definitions.

Attention bounds: tests/paged_rows.py.  The write: with u = 2^-24 the norm's factor is off by
at most 20 u (16 additions of a lane, 5 halving steps and the mean's product, halved by the
root, eps, a rsqrt of 4 u), two products more, a rotation by 2 u of |x_a| + |x_b|: 24 u of
the magnitudes, and half a step of the store.  Gathered rows, rows without a norm and parts
without a rotation are bit copies."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from tests.gpu_helpers import i32, lib
from tests.paged_rows import DT, Pages, assert_rows, chain_or_tree, f64, starts, words_of

pytestmark = pytest.mark.gpu
P = 64
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pa():
    return lib()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def normal(g, *shape, dt):
    return torch.from_numpy(g.normal(size=shape)).to(dt).cuda()


# ------------------------------------------------------------------------- absorbed form

class Batch:
    def __init__(self, lens, counts, H, R, bs, dt, kind="tree", seed=0):
        g = np.random.default_rng(seed + R + bs)
        self.lens, self.counts, self.H, self.R, self.dt = lens, counts, H, R, DT[dt]
        self.p = Pages(lens, bs, g)
        self.pool = self.p.pool((R + P,), self.dt, g)
        self.T = sum(counts)
        self.q = normal(g, self.T, H, R + P, dt=self.dt)
        self.out = torch.full((self.T, H, R), 7.0, dtype=self.dt, device="cuda")
        self.starts = starts(counts)
        self.W = -(-max(counts + [1]) // 32)
        self.mask = None
        if kind not in ("causal", "one"):
            self.mask = np.concatenate([words_of(chain_or_tree(n, kind, g), self.W)
                                        for n in counts if n] or [np.zeros((0, self.W), np.int32)])
        self.q_start = None if kind == "one" else i32(self.starts)
        self.scale = (128 + P) ** -0.5
        self.terms = 2 if max(counts + [0]) * H <= 32 else 1

    def run(self, pa, **kw):
        kw = dict(dict(q_start=self.q_start, max_q_len=max(self.counts + [1]),
                       tree_mask=None if self.mask is None else i32(self.mask),
                       max_seq_len=max(self.lens + [0])), **kw)
        pa.pa_latent_decode(self.out, self.q, self.pool, i32(self.p.tables), i32(self.lens),
                            self.scale, **kw)
        return self

    def check(self, skip=(), heads=None):
        got, q, pool = f64(self.out), f64(self.q), f64(self.pool)
        for b, (L, n) in enumerate(zip(self.lens, self.counts)):
            mine = slice(self.starts[b], self.starts[b] + n)
            if b in skip:
                assert (got[mine] == 7.0).all(), b
                continue
            if L == 0:
                assert (got[mine] == 0).all()
                continue
            seen = ol.visible(n, L, None if self.mask is None else self.mask[mine])
            x = self.p.rows(pool, b)
            for h in heads or range(self.H):
                ref = ol.attend(q[mine, h], x, x[:, :self.R], seen, self.scale)
                assert_rows(got[mine, h], *ref, self.R + P, self.dt, self.terms, (b, h))


DECODE = [
    # lens, new tokens, heads, latent, bs, type, what they hang on
    ([1], [1], 1, 256, 8, "fp16", "one"),
    ([5, 0, 64, 65, 1], [1] * 5, 16, 512, 16, "bf16", "one"),
    ([63, 64, 130, 200], [1] * 4, 128, 512, 16, "bf16", "one"),
    ([63, 128, 129, 700], [1] * 4, 128, 256, 64, "fp16", "one"),
    ([300, 17], [1] * 2, 40, 512, 32, "fp16", "one"),
    ([90, 33], [1] * 2, 96, 512, 16, "bf16", "one"),
    ([70, 300, 9], [3, 1, 9], 16, 512, 64, "bf16", "tree"),
    ([70, 300], [33, 40], 8, 256, 8, "bf16", "tree"),
    ([150, 66, 200], [66, 66, 5], 3, 512, 16, "bf16", "causal"),
    ([140], [12], 32, 512, 16, "fp16", "chain"),
    ([129, 0, 3], [4, 0, 3], 20, 256, 16, "fp16", "star"),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[2]}x{c[3]}-{c[5]}-{c[6]}")
def test_decode_parity(pa, case):
    Batch(*case).run(pa).check()


@pytest.mark.parametrize("H,R,n,dt", [(16, 512, 1, "bf16"), (128, 512, 1, "bf16"),
                                      (8, 256, 3, "fp16")])
def test_decode_split_over_the_length(pa, H, R, n, dt):
    b = Batch([7000, 3, 15001, 150], [n, min(n, 3), n, n], H, R, 16, dt)
    b.run(pa).check(heads=[0, H // 2, H - 1])


def test_decode_many_sequences(pa):
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 150, size=300)]
    Batch(lens, [1] * 300, 16, 256, 16, "bf16", "one").run(pa).check(heads=[0, 15])


def test_decode_rows_that_see_nothing(pa):
    b = Batch([6, 40], [6, 6], 8, 512, 16, "bf16")
    b.mask[2] = 0
    b.mask[8] = 0
    b.run(pa).check()
    assert (f64(b.out)[2] == 0).all()


@pytest.mark.parametrize("H", [4, 64])
def test_decode_scores_far_apart(pa, H):
    b = Batch([1500, 300], [1, 1], H, 512, 16, "bf16")
    for s in range(2):
        for t in range(0, b.lens[s], 97):
            b.pool[b.p.tables[s, t // 16], t % 16] *= 1 + t / 40
    b.run(pa).check(heads=[0, 1, H - 1])


def test_decode_unseen_rows_have_no_part(pa):
    b = Batch([70, 150, 6], [6, 20, 6], 4, 512, 16, "bf16", "star")
    for s, i, c, x in ((0, 1, 0, float("inf")), (1, 3, 511, float("nan")),
                       (1, 17, 512, float("nan")), (2, 4, 40, float("-inf"))):
        t = b.lens[s] - b.counts[s] + i
        b.pool[b.p.tables[s, t // 16], t % 16, c] = x
    b.run(pa).check()


def test_decode_bad_data(pa):
    b = Batch([40, 50, 60], [4, 5, 6], 8, 512, 16, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.run(pa, max_q_len=5, status=status)
    assert int(status) == 5
    b.check(skip=(2,))
    b.out.fill_(7.0)
    status.zero_()
    spare = [i for i in range(b.p.NB) if i not in b.p.tables]
    b.p.tables[1, 2] = b.p.NB + 5
    b.run(pa, status=status)
    assert int(status) == 5
    b.pool[spare[0]] = 0
    b.p.tables[1, 2] = spare[0]
    b.check()


@pytest.mark.parametrize("H", [65, 130, 200])
def test_decode_heads_that_do_not_fill_a_group(pa, H):
    Batch([200, 7, 300], [2, 1, 3], H, 256, 16, "bf16").run(pa).check(heads=[0, 63, 64, H - 1])


def test_decode_a_bound_whose_costs_pass_32_bits(pa):
    g = np.random.default_rng(8)
    lens = [int(x) for x in g.integers(0, 900, size=70)]
    b = Batch(lens, [1] * 70, 128, 512, 16, "bf16", "one")
    assert 70 * 4 * ((1 << 30) // 64) > 1 << 31
    b.run(pa, max_seq_len=(1 << 30) - 1).check(heads=[0, 100])


def test_decode_graph_replay_and_stream(pa):
    b = Batch([3000, 900, 0], [1] * 3, 128, 512, 16, "bf16", "one")
    s = torch.cuda.Stream()
    ws = pa.workspace_for_latent(b.out, b.pool)
    tables, lens = i32(b.p.tables), i32(b.lens)

    def step():
        pa.pa_latent_decode(b.out, b.q, b.pool, tables, lens, b.scale, max_seq_len=3000,
                            workspace=ws)
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    b.q.neg_()
    b.out.fill_(7.0)
    g.replay()
    first = b.out.clone()
    g.replay()
    torch.cuda.synchronize()
    b.check(heads=[0, 70, 127])
    assert torch.equal(first, b.out)


# ------------------------------------------------------------------------- the cache write

@pytest.mark.parametrize("lens,new,H,R,bs,dt,interleaved,norm,wide,positions", [
    ([5, 0, 64, 17], None, 16, 512, 16, "bf16", False, True, True, False),
    ([1], None, 1, 256, 8, "fp16", True, False, False, False),
    ([40, 7, 130], [40, 3, 77], 33, 512, 16, "bf16", True, True, True, False),
    ([40, 7, 130], [0, 7, 130], 5, 256, 64, "fp16", False, True, False, True),
    ([700, 900], [700, 900], 8, 512, 32, "bf16", False, True, True, True),
])
def test_append(pa, lens, new, H, R, bs, dt, interleaved, norm, wide, positions):
    g = np.random.default_rng(R + bs)
    dt = DT[dt]
    p = Pages(lens, bs, g)
    pool = p.pool((R + P,), dt, g)
    before = pool.clone()
    counts = [1] * len(lens) if new is None else new
    behind = 0 if new is None else 2
    T = sum(counts) + behind
    x = normal(g, T, R + P + (24 if wide else 0), dt=dt) * 3
    lat, key = x[:, :R], x[:, R:R + P]
    q = normal(g, T, H, 128 + P, dt=dt)[..., 128:]
    if not wide:
        lat, key, q = lat.contiguous(), key.contiguous(), q.contiguous()
    full = torch.full((T, H, R + P if wide else P), 7.0, dtype=dt, device="cuda")
    out = full[..., -P:]
    w = torch.from_numpy(g.uniform(0.5, 1.5, R)).to(dt).cuda() if norm else None
    th = g.uniform(-np.pi, np.pi, size=(max(lens) + 9, P // 2))
    cs = torch.from_numpy(np.concatenate([np.cos(th), np.sin(th)], 1)).float().cuda()
    pos = i32(g.integers(0, max(lens) + 9, size=T)) if positions else None
    pa.pa_latent_append(pool, lat, key, cs, i32(p.tables), i32(lens),
                        q_start=None if new is None else i32(starts(counts)), weight=w, eps=1e-5,
                        interleaved=interleaved, positions=pos, q_rope=q, q_out=out)
    half = torch.finfo(dt).eps / 2
    tiny = float(torch.finfo(dt).smallest_normal) * half
    lat64, key64, q64, cs64 = f64(lat), f64(key), f64(q), f64(cs)
    got, qgot, old = f64(pool), f64(out), bits(before)
    one, two = (slice(0, P, 2), slice(1, P, 2)) if interleaved else \
        (slice(0, P // 2), slice(P // 2, P))

    def turned(v, row):
        c, s = cs64[row, :P // 2], cs64[row, P // 2:]
        y, e = np.empty_like(v), np.empty_like(v)
        y[..., one], y[..., two] = v[..., one] * c - v[..., two] * s, v[..., two] * c + v[..., one] * s
        e[..., one] = e[..., two] = np.abs(v[..., one]) + np.abs(v[..., two])
        return y, e

    def close(a, ref, mag, what):
        bad = np.abs(a - ref) > half * (np.abs(ref) + 24 * U * mag) + 24 * U * mag + tiny
        assert not bad.any(), (what, int(bad.sum()))
    written = np.zeros((p.NB, bs), dtype=bool)
    t = 0
    for b, (L, n) in enumerate(zip(lens, counts)):
        if new is None and L == 0:
            assert (qgot[t] == 7.0).all()
            t += 1
            continue
        for i in range(n):
            at = L - n + i
            row = int(pos[t]) if positions else at
            slot = p.tables[b, at // bs], at % bs
            written[slot] = True
            ref = lat64[t]
            if norm:
                ref = ref / np.sqrt((ref * ref).mean() + 1e-5) * f64(w)
                close(got[slot][:R], ref, np.abs(ref), "norm")
            else:
                assert np.array_equal(got[slot][:R], ref)
            close(got[slot][R:], *turned(key64[t], row), "key")
            close(qgot[t], *turned(q64[t], row), "q")
            t += 1
    assert np.array_equal(bits(pool)[~written], old[~written])     # other rows untouched
    assert behind == 0 or (qgot[t:] == 7.0).all()
    if wide:
        assert (full[..., :R] == 7.0).all()                        # nor other columns


def test_append_without_rotation_copies(pa):
    g = np.random.default_rng(1)
    p = Pages([40, 9], 16, g)
    pool = p.pool((256 + P,), torch.bfloat16, g)
    x = normal(g, 49, 256 + P, dt=torch.bfloat16)
    q = normal(g, 49, 3, P, dt=torch.bfloat16)
    out = torch.zeros_like(q)
    pa.pa_latent_append(pool, x[:, :256], x[:, 256:], None, i32(p.tables), i32([40, 9]),
                        q_start=i32([0, 40, 49]), q_rope=q, q_out=out)
    rows = np.concatenate([p.rows(bits(pool), b) for b in range(2)])
    assert np.array_equal(rows, bits(x)) and torch.equal(out, q)


def test_append_in_place_and_beside(pa):
    """q_out may be q_rope itself, or other columns of the same rows; overlaps are refused."""
    g = np.random.default_rng(2)
    p = Pages([30], 16, g)
    pool = p.pool((256 + P,), torch.bfloat16, g)
    x = normal(g, 30, 256 + P, dt=torch.bfloat16)
    wide = normal(g, 30, 4, 3 * P, dt=torch.bfloat16)
    cs = pa.rope_table(30, P)
    src = wide[..., :P].clone()

    def f(q, out):
        pa.pa_latent_append(pool, x[:, :256], x[:, 256:], cs, i32(p.tables), i32([30]),
                            q_start=i32([0, 30]), q_rope=q, q_out=out)
    want = torch.empty_like(src)
    f(src, want)
    f(wide[..., :P], wide[..., P:2 * P])
    assert torch.equal(wide[..., P:2 * P], want)
    f(wide[..., :P], wide[..., :P])
    assert torch.equal(wide[..., :P], want)
    for lo in (8, P - 8):
        with pytest.raises(pa.PagedAttnError):
            f(wide[..., :P], wide[..., lo:lo + P])
    with pytest.raises(pa.PagedAttnError):
        f(wide[..., :P], x.view(-1)[:wide[..., :P].numel()].view(30, 4, P)
          if x.numel() >= wide[..., :P].numel() else x[:, :4 * P].view(30, 4, P))


def test_append_bad_data(pa):
    g = np.random.default_rng(3)
    p = Pages([30, 20, 40, 9], 16, g)
    pool = p.pool((256 + P,), torch.bfloat16, g)
    before = bits(pool)
    n = [4, 5, 6, 2]
    x = normal(g, 17, 256 + P, dt=torch.bfloat16)
    q, out = normal(g, 17, 3, P, dt=torch.bfloat16), torch.full((17, 3, P), 7.0).bfloat16().cuda()
    cs = pa.rope_table(34, P)                          # sequence 2's rows lie behind it
    tables = p.tables.copy()
    tables[0, 1] = -1                                  # sequence 0: no block for its new rows
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_latent_append(pool, x[:, :256], x[:, 256:], cs, i32(tables), i32([30, 3, 40, 9]),
                        q_start=i32(starts(n)), q_rope=q, q_out=out, status=status)
    assert int(status) == 5
    got = bits(pool)
    slot = p.tables[3, 0]
    changed = (got != before).any(-1)
    assert changed[slot, 7:9].all() and changed.sum() == 2     # sequence 3's two rows alone
    o = f64(out)
    assert (o[4:15] == 7.0).all() and (o[:4] != 7.0).any() and (o[15:] != 7.0).any()


# ------------------------------------------------------------------------- gather

@pytest.mark.parametrize("lens,n,R,bs,dt,stride", [
    ([50, 7, 23], [50, 7, 23], 256, 8, "fp16", 0),
    ([300, 0, 129, 1], [300, 0, 100, 1], 512, 16, "bf16", 8),
    ([64], [33], 512, 64, "bf16", 64),
])
def test_gather(pa, lens, n, R, bs, dt, stride):
    g = np.random.default_rng(R)
    p = Pages(lens, bs, g)
    pool = p.pool((R + P,), DT[dt], g)
    S = sum(n)
    full = torch.full((S + 3, R + P + stride), 7.0, dtype=DT[dt], device="cuda")
    out = full[:, :R + P]
    pa.pa_latent_gather(out, pool, i32(p.tables), i32(lens), i32(starts(n)))
    want = np.concatenate([p.rows(bits(pool), b)[:k] for b, k in enumerate(n)])
    assert np.array_equal(bits(out)[:S], want)
    assert (full[S:] == 7.0).all() and (full[:, R + P:] == 7.0).all()


def test_gather_bad_data(pa):
    g = np.random.default_rng(4)
    p = Pages([40, 30, 20], 16, g)
    pool = p.pool((256 + P,), torch.bfloat16, g)
    tables = p.tables.copy()
    tables[2, 1] = p.NB
    out = torch.full((90, 256 + P), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_latent_gather(out, pool, i32(tables), i32([40, 29, 20]), i32([0, 40, 70, 90]),
                        status=status)
    assert int(status) == 5
    o = bits(out)
    assert np.array_equal(o[:40], p.rows(bits(pool), 0))
    assert (out[40:70] == 7.0).all()
    assert np.array_equal(o[70:86], p.rows(bits(pool), 2)[:16]) and (o[86:] == 0).all()
    with pytest.raises(pa.PagedAttnError):                     # into the pool itself
        pa.pa_latent_gather(pool.view(-1, 256 + P)[:90], pool, i32(tables), i32([40, 29, 20]),
                            i32([0, 40, 70, 90]))


# ------------------------------------------------------------------------- expanded form

class Prompts:
    def __init__(self, lens, counts, H, dt, wide=True, seed=0):
        g = np.random.default_rng(seed + H)
        self.lens, self.counts, self.H, self.dt = lens, counts, H, DT[dt]
        self.S, self.T = sum(lens), sum(counts)
        self.kv = normal(g, self.S, H, 256, dt=self.dt)
        self.k = normal(g, self.S, 192 + P if wide else P, dt=self.dt)[:, -P:]
        self.q = normal(g, self.T, H, 128 + P, dt=self.dt)
        self.out = torch.full((self.T, H, 128), 7.0, dtype=self.dt, device="cuda")
        self.qs, self.ks = starts(counts), starts(lens)
        self.scale = (128 + P) ** -0.5

    def run(self, pa, **kw):
        kw.setdefault("max_q_len", max(self.counts))
        pa.pa_latent_prefill(self.out, self.q, self.kv, self.k, i32(self.qs), i32(self.ks),
                             self.scale, **kw)
        return self

    def check(self, skip=(), heads=None):
        got, q, kv, k = f64(self.out), f64(self.q), f64(self.kv), f64(self.k)
        for b, (L, n) in enumerate(zip(self.lens, self.counts)):
            mine, rows = slice(self.qs[b], self.qs[b] + n), slice(self.ks[b], self.ks[b] + L)
            if b in skip:
                assert (got[mine] == 7.0).all(), b
                continue
            for h in heads or range(self.H):
                key = np.concatenate([kv[rows, h, :128], k[rows]], 1)
                ref = ol.attend(q[mine, h], key, kv[rows, h, 128:], ol.visible(n, L), self.scale)
                assert_rows(got[mine, h], *ref, 192, self.dt, 1, (b, h))


@pytest.mark.parametrize("lens,counts,H,dt", [
    ([1], [1], 1, "fp16"),
    ([5, 128, 129], [5, 128, 129], 3, "bf16"),
    ([127, 300, 64], [127, 300, 64], 4, "fp16"),
    ([700, 33], [130, 1], 2, "bf16"),
    ([257, 513, 1], [256, 1, 1], 5, "bf16"),
    ([640, 0, 90], [255, 0, 90], 1, "bf16"),
])
def test_prefill_parity(pa, lens, counts, H, dt):
    Prompts(lens, counts, H, dt).run(pa).check()


def test_prefill_long(pa):
    Prompts([3000, 1111], [3000, 500], 4, "bf16", wide=False).run(pa).check(heads=[0, 3])


def test_prefill_scores_far_apart(pa):
    b = Prompts([900], [900], 2, "bf16")
    b.kv[::97, :, :128] *= torch.linspace(1, 30, 10, device="cuda", dtype=b.dt)[:, None, None]
    b.run(pa).check()


def test_prefill_unseen_tokens_have_no_part(pa):
    """Infinities and NaN reach the rows that see them, and rows behind a sequence no one."""
    b = Prompts([300, 140], [300, 140], 2, "bf16")
    b.kv[200, 0, 130] = float("inf")
    b.kv[250, 1, 3] = float("nan")
    b.kv[300, 1, 200] = float("nan")                  # the next sequence's first token
    b.k[300 + 77, 5] = float("inf")
    b.run(pa).check()


def test_prefill_bad_sequences(pa):
    b = Prompts([40, 50, 60], [40, 5, 60], 2, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.run(pa, max_q_len=59, status=status)
    assert int(status) == 5
    b.check(skip=(2,))
    b.out.fill_(7.0)
    status.zero_()
    ks = b.ks.copy()
    ks[1:] = [39, 90, 150]                             # sequence 0: fewer keys than queries
    pa.pa_latent_prefill(b.out, b.q, b.kv, b.k, i32(b.qs), i32(ks), b.scale, max_q_len=60,
                         status=status)
    assert int(status) == 5
    assert (b.out[:40] == 7.0).all() and not (b.out[45:] == 7.0).all()


def test_prefill_rows_behind_stay(pa):
    b = Prompts([40, 50], [40, 50], 2, "bf16")
    out = torch.full((96, 2, 128), 7.0, dtype=b.dt, device="cuda")
    pa.pa_latent_prefill(out, torch.cat([b.q, b.q[:6]]), torch.cat([b.kv, b.kv[:9]]),
                         torch.cat([b.k, b.k[:9]]), i32(b.qs), i32(b.ks), b.scale, max_q_len=50)
    assert (out[90:] == 7.0).all()
    b.out = out[:90]
    b.check()


# ------------------------------------------------------------------------- together

def test_a_serving_run(pa):
    """Prompts written, a second chunk over the cached prefix in the expanded form, then a
    drafted tree and a single token in the absorbed form: each equals attention over all of the
    sequence's own rows, in 64 bits."""
    g = np.random.default_rng(9)
    dt, R, H, bs = torch.bfloat16, 256, 4, 16
    first, chunk, tree = [37, 90], [30, 17], [5, 9]
    lens = [a + b for a, b in zip(first, chunk)]
    total = [a + b for a, b in zip(lens, tree)]
    p = Pages(total, bs, g)
    pool = p.pool((R + P,), dt, g)
    cs = pa.rope_table(256, P)
    wk, wv = normal(g, H, 128, R, dt=dt) * 0.1, normal(g, H, 128, R, dt=dt) * 0.1
    weight = torch.from_numpy(g.uniform(0.5, 1.5, R)).to(dt).cuda()
    tables = i32(p.tables)

    def write(upto, n, positions=None):
        T = sum(n)
        x, q = normal(g, T, R + P, dt=dt), normal(g, T, H, 128 + P, dt=dt)
        pa.pa_latent_append(pool, x[:, :R], x[:, R:], cs, tables, i32(upto), q_start=i32(starts(n)),
                            weight=weight, positions=positions, q_rope=q[..., 128:],
                            q_out=q[..., 128:])
        return q

    def absorbed(q):
        qa = torch.einsum("thd,hdr->thr", q[..., :128].float(), wk.float()).to(dt)
        return torch.cat([qa, q[..., 128:]], 2).contiguous()

    write(first, first)
    q = write(lens, chunk)
    rows = torch.empty(sum(lens), R + P, dtype=dt, device="cuda")
    pa.pa_latent_gather(rows, pool, tables, i32(lens), i32(starts(lens)))
    expand = torch.cat([wk, wv], 1)                                    # [H, 256, R]
    kv = torch.einsum("sr,hdr->shd", rows[:, :R].float(), expand.float()).to(dt).contiguous()
    out = torch.empty(sum(chunk), H, 128, dtype=dt, device="cuda")
    scale = (128 + P) ** -0.5
    pa.pa_latent_prefill(out, q, kv, rows[:, R:], i32(starts(chunk)), i32(starts(lens)), scale)
    qn, kvn, rn, on = f64(q), f64(kv), f64(rows), f64(out)
    for b in range(2):
        mine, at = slice(*starts(chunk)[b:b + 2]), slice(*starts(lens)[b:b + 2])
        assert np.array_equal(rn[at], p.rows(f64(pool), b)[:lens[b]])
        for h in range(H):
            ref = ol.attend(qn[mine, h], np.concatenate([kvn[at, h, :128], rn[at, R:]], 1),
                            kvn[at, h, 128:], ol.visible(chunk[b], lens[b]), scale)
            assert_rows(on[mine, h], *ref, 192, dt, 1, ("prefill", b, h))
    parents = [chain_or_tree(n, "tree", g) for n in tree]
    depth = []
    for b, ps in enumerate(parents):
        d = []
        for x in ps:
            d.append(d[x] + 1 if x >= 0 else 0)
        depth += [lens[b] + x for x in d]
    q = absorbed(write(total, tree, i32(depth)))
    out = torch.empty(sum(tree), H, R, dtype=dt, device="cuda")
    mask = pa.tree_mask(parents)
    pa.pa_latent_decode(out, q, pool, tables, i32(total), scale, q_start=i32(starts(tree)),
                        tree_mask=mask)
    qn, on, words = f64(q), f64(out), mask.cpu().numpy()
    for b in range(2):
        mine = slice(*starts(tree)[b:b + 2])
        x = p.rows(f64(pool), b)
        for h in range(H):
            ref = ol.attend(qn[mine, h], x, x[:, :R], ol.visible(tree[b], total[b], words[mine]),
                            scale)
            # nine new tokens of four heads are 36 columns: weights of one term
            assert_rows(on[mine, h], *ref, R + P, dt, 1, ("tree", b, h))

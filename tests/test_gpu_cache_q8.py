"""GPU parity of the 8-bit cache's decode attention and expansion, and of a serving run
over it, against the fp64 oracle.

Bounds of the decode.  With p the softmax weights, A = sum_t p_t |V_t| per output element
and S = max_t scale sum_d |q_d K_td|:
  - a score sums at most 3 x 128 products in fp32: off by at most 384 * 2^-24 S = 2^-15.4 S
    (natural units), a weight by twice that (itself and the normaliser);
  - a weight may be held as three e4m3 digits of an fp16 number: fp16 has 11 bits, so half
    a step is 2^-11 of the weight, and the digits, 4 bits each, hold all 11; or 2^-25 of the
    largest weight where that is more (each token adds at most that much of |V|);
  - the sums and the join of splits: fp32, far below; taken as 2^-16 A;
  - the store: half a step of the type.
So |d| <= eps/2 |ref| + (2^-11 + 2^-14.4 S + 2^-16) A + n 2^-25 max|V| (n tokens) + half
a subnormal step."""
import numpy as np
import pytest
import torch

from oracle import cache_q8 as oq
from tests.gpu_helpers import i32, lib

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def pa():
    return lib()


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    def __init__(self, lens, G, H, D, bs, dt, seed=0, po2=True):
        g = np.random.default_rng(7 * seed + D + bs)
        self.lens, self.H, self.D, self.bs, self.dt = lens, H, D, bs, DT[dt]
        used = [-(-n // bs) for n in lens]
        self.NB = sum(used) + 3
        order = g.permutation(self.NB)
        self.tables = np.full((len(lens), max(used) + 2), 1 << 30, dtype=np.int32)
        at = 0
        live = np.zeros((self.NB, bs), dtype=bool)
        for b, n in enumerate(used):
            self.tables[b, :n] = order[at:at + n]
            at += n
            pos = np.arange(lens[b])
            live[self.tables[b, pos // bs], pos % bs] = True
        self.codes, self.scales = [], []
        for _ in range(2):
            x = g.normal(size=(self.NB, H, bs, D)) * 100
            c = oq.encode_e4m3(x)
            c.transpose(0, 2, 1, 3)[~live] = 0x7F          # NaN behind every sequence's end
            sc = 2.0 ** g.integers(-9, -4, size=(self.NB, H))
            if not po2:
                sc = sc * g.uniform(0.7, 1.4, size=sc.shape)
            sc = sc.astype(np.float32)
            sc[~live.any(1)] = np.nan                      # scales of blocks nobody holds
            self.codes.append(c)
            self.scales.append(sc)
        self.pools = [torch.from_numpy(c.copy()).cuda() for c in self.codes]
        self.sc = [torch.from_numpy(x.copy()).cuda() for x in self.scales]
        self.q = torch.from_numpy(g.normal(size=(len(lens), G * H, D))).to(self.dt).cuda()
        self.scale = float(np.float32(D ** -0.5))

    def check(self, out, lens=None, rows=None):
        k, v = (oq.values_q8(c, s) for c, s in zip(self.codes, self.scales))
        check_decode(f64(out), f64(self.q), k, v, self.tables, lens or self.lens, self.scale,
                     self.dt, rows)

    def run(self, pa, **kw):
        out = torch.full_like(self.q, float("nan"))
        lens = kw.pop("lens", self.lens)
        pa.pa_decode_q8(out, self.q, *self.pools, *self.sc, i32(kw.pop("tables", self.tables)),
                        i32(lens), self.scale, **kw)
        torch.cuda.synchronize()
        return out


def check_decode(got, q, k, v, tables, lens, scale, dt, rows=None):
    half = torch.finfo(dt).eps / 2
    tiny = float(torch.finfo(dt).smallest_normal) * half
    for b in rows if rows is not None else range(len(lens)):
        ref, mass, size = oq.decode_with_spread(q[b], k, v, tables[b], lens[b], scale)
        if lens[b] == 0:
            assert not got[b].any()
            continue
        pos = np.arange(lens[b])
        blk = np.asarray(tables[b], dtype=np.int64)[pos // k.shape[1]]
        top = np.abs(v[blk, pos % k.shape[1]]).max()
        e = (2.0 ** -11 + 2.0 ** -14.4 * size[:, None] + 2.0 ** -16) * mass + \
            lens[b] * 2.0 ** -25 * top
        bad = ~(np.abs(got[b] - ref) <= half * (np.abs(ref) + e) + e + tiny)
        assert not bad.any(), (b, lens[b], int(bad.sum()), np.argwhere(bad)[:3],
                               np.abs(got[b] - ref).max())


LENS = [0, 1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 640, 1000]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("D,G,H", [(64, 1, 4), (64, 4, 2), (64, 7, 1), (64, 16, 1), (128, 1, 3),
                                   (128, 2, 2), (128, 4, 2), (128, 5, 1), (128, 8, 1),
                                   (128, 16, 1)])
def test_decode(pa, D, G, H, bs, dt):
    b = Batch(LENS, G, H, D, bs, dt, seed=G)
    b.check(b.run(pa))


@pytest.mark.parametrize("D,G,H", [(128, 3, 1), (128, 6, 2), (128, 7, 1), (128, 10, 1),
                                   (128, 12, 1), (128, 20, 1), (128, 33, 1), (64, 3, 2),
                                   (64, 20, 1)])
def test_decode_other_groups(pa, D, G, H):
    b = Batch([1, 130, 400], G, H, D, 16, "bf16", seed=G)
    b.check(b.run(pa))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[9001], [5000, 1, 4097, 0, 12]])
def test_decode_long_sequences_are_split(pa, D, lens):
    b = Batch(lens, 4, 2, D, 16, "fp16", seed=3)
    b.check(b.run(pa))


def test_decode_many_sequences(pa):
    lens = [(37 * i) % 200 for i in range(700)]
    b = Batch(lens, 4, 2, 128, 16, "bf16", seed=4)
    out = b.run(pa)
    b.check(out, rows=range(0, 700, 9))


@pytest.mark.parametrize("D,G,bs", [(128, 8, 32), (128, 16, 16), (128, 5, 64), (128, 1, 8), (64, 4, 16),
                                    (64, 8, 8)])
def test_decode_many_tiles_per_window(pa, D, G, bs):
    """Tens of tiles to every CTA: the rings and buffers go round many times.  Against the
    definition in fp64, by torch on the GPU, for some heads of each sequence."""
    H, lens = 8, [70001, 20000, 31, 45678, 3000, 1]
    g = torch.Generator("cuda").manual_seed(D + G)
    used = [-(-n // bs) for n in lens]
    NB = sum(used) + 3
    order = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(used):
        tables[b, :n] = order[sum(used[:b]):sum(used[:b + 1])]
    pools = [torch.empty(NB, H, bs, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    for p in pools:
        for i in range(0, NB, 1024):       # normal values, 100 times
            x = torch.randn(min(1024, NB - i), H, bs, D, generator=g, device="cuda") * 100
            p[i:i + 1024] = x.clamp(-448, 448).to(pa.E4M3).view(torch.uint8)
    sc = [torch.exp2(torch.randint(-9, -5, (NB, H), generator=g, device="cuda").float())
          for _ in "kv"]
    q = torch.randn(len(lens), G * H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_q8(out, q, *pools, *sc, tables, i32(lens), 0.05, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for b, n in enumerate(lens):
        blk = tables[b, :used[b]].long()
        for h in (0, 3, H - 1):
            k, v = ((p[blk, h].view(pa.E4M3).double() * s[blk, h].double()[:, None, None])
                    .reshape(-1, D)[:n] for p, s in zip(pools, sc))
            mine = slice(h * G, (h + 1) * G)
            qd = q[b, mine].double()
            w = torch.softmax(0.05 * qd @ k.T, -1)
            ref, mass = w @ v, w @ v.abs()
            size = 0.05 * (qd.abs() @ k.abs().T).amax(-1, keepdim=True)
            e = (2.0 ** -11 + 2.0 ** -14.4 * size + 2.0 ** -16) * mass + n * 2.0 ** -25 * v.abs().max()
            bad = ~((out[b, mine].double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + e) + e)
            assert not bad.any(), (b, h, int(bad.sum()))


@pytest.mark.parametrize("D,G,n", [(128, 1, 40001), (128, 3, 6500), (128, 5, 40001), (128, 9, 40001),
                                   (64, 7, 80003)])
def test_decode_one_item_in_many_parts(pa, D, G, n):
    """One KV head and one sequence: every window boundary cuts the same item(s)."""
    b = Batch([n], G, 1, D, 32, "bf16", seed=G)
    b.check(b.run(pa))


@pytest.mark.parametrize("G", [1, 8])
def test_decode_d64_segments_of_one_tile(pa, G):
    """head_dim 64: segments of one tile follow one another to the end of every window, and
    each hands the sums of odd tokens to the threads of even ones."""
    lens = [1 + (61 * i) % 256 for i in range(500)]
    b = Batch(lens, G, 3, 64, 16, "bf16", seed=G)
    outs = [b.run(pa) for _ in range(6)]
    b.check(outs[0], rows=range(0, 500, 3))
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs)


def test_decode_any_positive_scale(pa):
    b = Batch([300, 77], 4, 2, 128, 16, "bf16", seed=5, po2=False)
    b.check(b.run(pa))


def test_decode_scales_far_apart(pa):
    """Blocks of one sequence whose scales differ by 2^40: the large values decide."""
    b = Batch([200], 4, 1, 128, 16, "bf16", seed=6)
    blk = b.tables[0]
    for i, e in enumerate([-30, 10, -8, 3, -64, 0, -20]):
        b.scales[1][blk[i]] = 2.0 ** e
    b.sc[1].copy_(torch.from_numpy(b.scales[1]))
    b.check(b.run(pa))


def test_decode_nan_in_a_live_row_reaches_only_its_heads(pa):
    b = Batch([100, 100], 4, 2, 128, 16, "bf16", seed=7)
    ok = b.run(pa)
    b.pools[0][b.tables[0, 2], 1, 3, 5] = 0x7F
    out = b.run(pa)
    assert torch.isnan(out[0, 4:]).all()
    assert torch.equal(out[0, :4], ok[0, :4]) and torch.equal(out[1], ok[1])


def test_decode_length_bounds(pa):
    """A length past max_seq_len is cut to it and reported; a negative one is empty."""
    b = Batch([64, 100, 40], 4, 2, 128, 16, "bf16", seed=8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.run(pa, lens=[64, 100, -3], max_seq_len=90, status=status)
    assert int(status.item()) == 5
    b.check(out, lens=[64, 90, 0])


def test_decode_bad_block_reads_zeros(pa):
    b = Batch([100, 50], 4, 2, 128, 16, "bf16", seed=9)
    for bad in (b.NB, -1, 1 << 30, -(1 << 31)):
        tables = b.tables.copy()
        tables[0, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = b.run(pa, tables=tables, status=status)
        assert int(status.item()) == 5
        c = [np.concatenate([x, np.zeros_like(x[:1])]) for x in b.codes]
        s = [np.concatenate([x, np.ones_like(x[:1])]) for x in b.scales]
        tables[0, 3] = b.NB                         # a block of zeros, to the oracle
        check_decode(f64(out), f64(b.q), oq.values_q8(c[0], s[0]), oq.values_q8(c[1], s[1]),
                     tables, b.lens, b.scale, b.dt)


def test_decode_repeats_to_the_bit_whatever_the_workspace_holds(pa):
    b = Batch([3000, 5, 0, 800], 4, 2, 128, 16, "bf16", seed=10)
    mx = 3000
    ws = pa.workspace_for_q8(b.q, b.pools[0], mx)
    outs = []
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        outs.append(b.run(pa, workspace=ws, max_seq_len=mx).view(torch.int16))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    wide = b.run(pa).view(torch.int16)              # max_seq_len only bounds
    assert torch.equal(wide[2], outs[0][2])
    b.check(wide.view(b.dt))


def test_decode_two_graphs_share_a_workspace(pa):
    """Captured calls of two batches over one workspace, replayed in turn on one stream."""
    a = Batch([2000, 30, 555], 4, 2, 128, 16, "bf16", seed=11)
    b = Batch([100, 4000], 5, 1, 128, 32, "bf16", seed=12)
    n = max(pa.workspace_for_q8(x.q, x.pools[0], 4000).numel() for x in (a, b))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x in (a, b):
        x.args = (*x.pools, *x.sc, i32(x.tables), i32(x.lens), x.scale)
        out = torch.zeros_like(x.q)
        pa.pa_decode_q8(out, x.q, *x.args, workspace=ws, max_seq_len=4000 if x is b else 2000)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode_q8(out, x.q, *x.args, workspace=ws, max_seq_len=4000 if x is b else 2000)
        graphs.append(g)
        outs.append(out)
    for out in outs:
        out.fill_(float("nan"))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


def test_decode_on_two_streams_at_once(pa):
    a = Batch([2000, 30, 555], 4, 2, 128, 16, "bf16", seed=13)
    b = Batch([100, 4000], 4, 2, 64, 32, "fp16", seed=14)
    outs = []
    for x in (a, b):
        x.s = torch.cuda.Stream()
        x.args = (*x.pools, *x.sc, i32(x.tables), i32(x.lens), x.scale)
        x.ws = pa.workspace_for_q8(x.q, x.pools[0], 4000)
        outs.append(torch.zeros_like(x.q))
    torch.cuda.synchronize()
    for _ in range(4):
        for x, out in zip((a, b), outs):
            pa.pa_decode_q8(out, x.q, *x.args, workspace=x.ws, max_seq_len=max(x.lens),
                            stream=x.s)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


def test_decode_offsets_past_32_bits(pa):
    """Codes past 2^32 bytes of the pool."""
    H, D, bs = 8, 128, 64
    NB = (1 << 32) // (H * D * bs) + 3
    k8, v8, ks, vs = pa.alloc_cache_q8(NB, H, bs, D)
    far = [NB - 1, 0, NB - 2]
    g = torch.Generator("cuda").manual_seed(1)
    for i in far:
        k8[i] = torch.randn(H, bs, D, generator=g, device="cuda").to(pa.E4M3)
        v8[i] = torch.randn(H, bs, D, generator=g, device="cuda").to(pa.E4M3)
    q = torch.randn(1, 4 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    pa.pa_decode_q8(out, q, k8, v8, ks, vs, i32([far]), i32([150]), 0.1)
    torch.cuda.synchronize()
    k, v = (f64(torch.stack([x[i].float() for i in far])).transpose(0, 2, 1, 3) for x in (k8, v8))
    check_decode(f64(out), f64(q), k, v, [[0, 1, 2]], [150], 0.1, torch.bfloat16)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("H,D,bs", [(1, 64, 8), (3, 128, 16), (8, 128, 16), (5, 64, 64),
                                    (2, 128, 32), (32, 128, 64)])
def test_expand(pa, H, D, bs, dt):
    g = np.random.default_rng(H + D + bs)
    NB, ND, n = 9, 12, 5
    codes = [g.integers(0, 256, size=(NB, H, bs, D)).astype(np.uint8) for _ in "kv"]
    sc = [(2.0 ** g.integers(-12, 9, size=(NB, H))).astype(np.float32) for _ in "kv"]
    pairs = np.stack([g.permutation(NB)[:n], g.permutation(ND)[:n]], 1)
    pools = [torch.full((ND, bs, H, D), 3.0, dtype=DT[dt], device="cuda") for _ in "kv"]
    pa.pa_expand_blocks_q8(*pools, *(torch.from_numpy(c).cuda() for c in codes),
                           *(torch.from_numpy(s).cuda() for s in sc), i32(pairs))
    torch.cuda.synchronize()
    for p, c, s in zip(pools, codes, sc):
        want = np.full((ND, bs, H, D), 3.0)
        most = torch.finfo(DT[dt]).max
        with np.errstate(invalid="ignore"):
            v = np.clip(oq.values_q8(c, s), -most, most)
        for src, dst in pairs:
            want[dst] = v[src]
        want = torch.from_numpy(want).to(DT[dt]).double().numpy()    # one rounding (fp16 only)
        got = f64(p)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_expand_bad_ids_are_reported_and_skipped(pa):
    k8, v8, ks, vs = pa.alloc_cache_q8(4, 2, 16, 64)
    k8.view(torch.uint8).fill_(0x38)                                # 1.0
    pools = [torch.zeros(3, 16, 2, 64, dtype=torch.float16, device="cuda") for _ in "kv"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pairs = i32([[4, 0], [0, 3], [-1, 1], [1, -1], [2, 2]])
    pa.pa_expand_blocks_q8(*pools, k8, v8, ks, vs, pairs, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 5
    assert (pools[0][2] == 1).all() and not pools[0][:2].any()


@pytest.mark.parametrize("H,G,D,bs,dt", [(4, 2, 128, 16, "bf16"), (4, 4, 64, 8, "fp16")])
def test_a_serving_run(pa, H, G, D, bs, dt):
    """Prompts are written rotated to the 8-bit cache, expanded and attended by pa_prefill;
    a block is cloned for a fork; then steps of one token each, written and attended.  The
    cache follows the oracle, and each attention matches the oracle over the cache."""
    g = np.random.default_rng(D)
    t_dt = DT[dt]
    prompts = [21, 40, 7]
    bm = pa.BlockManager(40, bs)
    seqs = [bm.new_sequence(n) for n in prompts]
    k8, v8, ks, vs = pa.alloc_cache_q8(40, H, bs, D)
    table = pa.rope_table(64, D, 500.0)
    qw, kw = (torch.from_numpy(g.uniform(0.5, 1.5, D)).to(t_dt).cuda() for _ in "qk")
    oracle = [np.zeros((40, H, bs, D), dtype=np.uint8), np.ones((40, H)),
              np.zeros((40, H, bs, D), dtype=np.uint8), np.ones((40, H))]
    scale = D ** -0.5

    def write(tables, lens, q_start):
        T = len(lens) if q_start is None else int(q_start[-1])
        qkv = torch.from_numpy(g.normal(size=(T, (G + 2) * H, D))).to(t_dt).cuda()
        q, k, v = qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
        out = torch.empty(T, G * H, D, dtype=t_dt, device="cuda")
        pa.pa_rope_append_q8(out, k8, v8, ks, vs, q, k, v, table, i32(tables), i32(lens),
                             q_start=None if q_start is None else i32(q_start), q_weight=qw,
                             k_weight=kw)
        places = oq.placements(lens, q_start, tables, bs)
        pos = np.array([p[2] for p in places])
        keys = oq.rotate(oq.rms_norm(f64(k), f64(kw), 1e-6), f64(table)[pos], False)
        oq.append_q8(oracle[0], oracle[1], keys, places)
        oq.append_q8(oracle[2], oracle[3], f64(v), places)
        return out

    def cache():
        """The GPU's cache, after a comparison with the oracle's: values to the bit; keys
        within a code step (their fp32 error may move a rounding)."""
        torch.cuda.synchronize()
        got = [k8.view(torch.uint8).cpu().numpy(), f64(ks), v8.view(torch.uint8).cpu().numpy(),
               f64(vs)]
        assert np.array_equal(got[2], oracle[2]) and np.array_equal(got[3], oracle[3])
        assert np.array_equal(got[1], oracle[1])
        a, b = oq.decode_e4m3(got[0]), oq.decode_e4m3(oracle[0])
        assert (np.abs(a - b) <= np.maximum(np.abs(b) * 2.0 ** -3, 2.0 ** -9)).all()
        assert (a != b).mean() < 1e-3
        oracle[0][:] = got[0]
        return oq.values_q8(got[0], got[1]), oq.values_q8(got[2], got[3])

    tables, lens = bm.export(seqs, 12, -1)
    q_start = np.concatenate([[0], np.cumsum(prompts)])
    q = write(tables.numpy(), lens.tolist(), q_start)
    used = sorted({int(x) for row in tables.numpy() for x in row if x >= 0})
    stage = {b: i for i, b in enumerate(used)}
    pools = [torch.zeros(len(used), bs, H, D, dtype=t_dt, device="cuda") for _ in "kv"]
    pa.pa_expand_blocks_q8(*pools, k8, v8, ks, vs, i32([[b, i] for b, i in stage.items()]))
    staged = np.array([[stage.get(int(x), 0) for x in row] for row in tables.numpy()])
    out = torch.empty_like(q)
    pa.pa_prefill(out, q, *pools, i32(staged), i32(lens.numpy()), i32(q_start), scale,
                  max_q_len=max(prompts))
    k, v = cache()
    got, qq = f64(out), f64(q)
    for b, n in enumerate(prompts):
        for i in range(n):
            ref = oq.decode_with_spread(qq[q_start[b] + i], k, v, tables[b].numpy(), i + 1, scale)[0]
            d = np.abs(got[q_start[b] + i] - ref)
            assert (d <= 2e-3 + 1e-2 * np.abs(ref)).all()      # pa_prefill's own acceptance

    seqs.append(bm.fork(seqs[0]))
    ws = None
    for _ in range(bs + 3):
        clones = [c for c in (bm.append(s)[1] for s in seqs) if c]
        if clones:
            pa.pa_copy_blocks_multi([k8, v8], i32(clones))
            pa.pa_copy_blocks_multi([ks, vs], i32(clones))
            for a, b in clones:
                for x in oracle:
                    x[b] = x[a]
        tables, lens = bm.export(seqs, 12, -1)
        q = write(tables.numpy(), lens.tolist(), None)
        out = torch.empty_like(q)
        ws = ws if ws is not None else pa.workspace_for_q8(q, k8, 12 * bs)
        pa.pa_decode_q8(out, q, k8, v8, ks, vs, i32(tables.numpy()), i32(lens.numpy()), scale,
                        max_seq_len=12 * bs, workspace=ws)
        k, v = cache()
        check_decode(f64(out), f64(q), k, v, tables.numpy(), lens.tolist(), scale, t_dt)

"""Argument checks of the drafted trees and the latent cache: every refusal comes back before
any launch (CPU only: no kernel runs)."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_301_gb300 import build
    build.build()
    from paged_kv_cache_301_gb300 import _lib
    return _lib.load()


# addresses far apart, so that nothing overlaps; no kernel runs
A = {n: (i + 1) << 40 for i, n in enumerate(
    "out q k_pool v_pool tables lens q_start mask ws pool latent key weight cos_sin positions "
    "q_rope q_out kv kv_start".split())}


def _tree(lib, **kw):
    a = dict(A, B=2, T=5, Hq=8, H=2, D=128, bs=16, MB=4, NB=8, mq=3, words=1, mx=64, scale=0.1,
             dtype=1, ws_bytes=1 << 40)
    a.update(kw)
    return lib.pa_decode_tree(
        a["out"], a["q"], a["k_pool"], a["v_pool"], a["tables"], a["lens"], a["q_start"],
        a["mask"], a["B"], a["T"], a["Hq"], a["H"], a["D"], a["bs"], a["MB"], a["NB"], a["mq"],
        a["words"], a["mx"], a["scale"], a["dtype"], a["ws"], a["ws_bytes"], None, None)


def _latent(lib, **kw):
    a = dict(A, B=2, T=5, Hq=8, R=512, P=64, bs=16, MB=4, NB=8, mq=3, words=1, mx=64, scale=0.1,
             dtype=1, ws_bytes=1 << 40)
    a.update(kw)
    return lib.pa_latent_decode(
        a["out"], a["q"], a["pool"], a["tables"], a["lens"], a["q_start"], a["mask"], a["B"],
        a["T"], a["Hq"], a["R"], a["P"], a["bs"], a["MB"], a["NB"], a["mq"], a["words"], a["mx"],
        a["scale"], a["dtype"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("f", [_tree, _latent], ids=["tree", "latent"])
def test_decode_refusals(lib, f):
    def g(**kw):
        return f(lib, **kw)
    assert g(bs=12) == 2 and g(dtype=5) == 2
    assert g(B=-1) == 1 and g(T=-1) == 1 and g(Hq=0) == 1 and g(mq=-1) == 1
    assert g(MB=0) == 1 and g(NB=0) == 1 and g(mx=-1) == 1 and g(mx=1 << 30) == 1
    assert g(NB=1 << 27) == 1                            # 2^31 rows
    assert g(scale=float("nan")) == 1 and g(scale=float("inf")) == 1
    assert g(mq=33) == 1 and g(words=0) == 1             # more new tokens than the mask has bits
    assert g(mq=65537, mask=None) == 1
    assert g(q_start=None) == 1                          # one row per sequence without it
    for p in ("out", "q", "tables", "lens"):
        assert g(**{p: None}) == 1, p
    for p in ("out", "q"):
        assert g(**{p: A[p] + 8}) == 1, p
    assert g(ws=None) == 3 and g(ws=A["ws"] + 16) == 3 and g(ws_bytes=0) == 3
    assert g(B=0, T=0) == 0 and g(T=0) == 0


def test_tree_refusals(lib):
    assert _tree(lib, D=96) == 2 and _tree(lib, Hq=7) == 1 and _tree(lib, H=0) == 1
    for p in ("k_pool", "v_pool"):
        assert _tree(lib, **{p: None}) == 1 and _tree(lib, **{p: A[p] + 8}) == 1
    f = lib.pa_decode_tree_workspace_bytes
    assert f(8, 2, 128, 4) > 0 and f(8, 2, 128, 4) % 256 == 0
    assert f(8, 3, 128, 4) == 0 and f(8, 2, 96, 4) == 0 and f(8, 2, 128, -1) == 0


def test_latent_decode_refusals(lib):
    assert _latent(lib, R=384) == 2 and _latent(lib, P=32) == 2
    assert _latent(lib, pool=None) == 1 and _latent(lib, pool=A["pool"] + 8) == 1
    f = lib.pa_latent_decode_workspace_bytes
    assert f(128, 512, 64, 1) > 0 and f(128, 512, 64, 1) % 256 == 0
    assert f(0, 512, 64, 1) == 0 and f(128, 500, 64, 1) == 0 and f(128, 512, 64, -1) == 0


def _append(lib, **kw):
    a = dict(A, eps=1e-6, mp=64, inter=0, positions=None, B=2, T=5, xs=0, ks=0, qs=0, qh=0, os=0,
             oh=0, Hq=8, R=512, P=64, bs=16, MB=4, NB=8, dtype=1)
    a.update(kw)
    return lib.pa_latent_append(
        a["pool"], a["latent"], a["key"], a["weight"], a["eps"], a["cos_sin"], a["mp"],
        a["inter"], a["positions"], a["q_rope"], a["q_out"], a["tables"], a["lens"],
        a["q_start"], a["B"], a["T"], a["xs"], a["ks"], a["qs"], a["qh"], a["os"], a["oh"],
        a["Hq"], a["R"], a["P"], a["bs"], a["MB"], a["NB"], a["dtype"], None, None)


def test_append_refusals(lib):
    def g(**kw):
        return _append(lib, **kw)
    assert g(R=500) == 2 and g(P=32) == 2 and g(bs=12) == 2 and g(dtype=5) == 2
    assert g(B=-1) == 1 and g(T=-1) == 1 and g(MB=0) == 1 and g(NB=0) == 1
    assert g(eps=-1.0) == 1 and g(eps=float("nan")) == 1 and g(eps=float("inf")) == 1
    assert g(mp=0) == 1 and g(q_start=None) == 1 and g(Hq=0) == 1
    assert g(q_out=None) == 1 and g(q_rope=None) == 1    # both or none
    for p in ("pool", "latent", "key", "tables", "lens"):
        assert g(**{p: None}) == 1, p
    for p in ("pool", "latent", "key", "weight", "cos_sin", "q_rope", "q_out"):
        assert g(**{p: A[p] + 8}) == 1, p
    assert g(xs=504) == 1 and g(xs=516) == 1 and g(ks=56) == 1 and g(ks=-8) == 1
    assert g(qh=56) == 1 and g(qh=68) == 1 and g(qs=504) == 1 and g(oh=32) == 1
    assert g(os=8 * 64 - 8) == 1
    assert g(q_out=A["q_rope"] + 16) == 1                # a shifted overlap
    assert g(q_out=A["q_rope"], os=1024) == 1            # in place with other strides
    assert g(q_out=A["latent"]) == 1 and g(q_out=A["key"] + 16) == 1
    assert g(B=0, T=0) == 0 and g(T=0) == 0


def _gather(lib, **kw):
    a = dict(A, B=2, S=50, os=0, R=512, P=64, bs=16, MB=4, NB=8, dtype=1)
    a.update(kw)
    return lib.pa_latent_gather(a["out"], a["pool"], a["tables"], a["lens"], a["kv_start"],
                                a["B"], a["S"], a["os"], a["R"], a["P"], a["bs"], a["MB"],
                                a["NB"], a["dtype"], None, None)


def test_gather_refusals(lib):
    def g(**kw):
        return _gather(lib, **kw)
    assert g(R=500) == 2 and g(P=32) == 2 and g(bs=12) == 2 and g(dtype=5) == 2
    assert g(B=-1) == 1 and g(S=-1) == 1 and g(MB=0) == 1 and g(NB=0) == 1
    assert g(os=568) == 1 and g(os=580) == 1
    for p in ("out", "pool", "tables", "lens", "kv_start"):
        assert g(**{p: None}) == 1, p
    assert g(out=A["out"] + 8) == 1 and g(pool=A["pool"] + 8) == 1
    assert g(out=A["pool"] + 16) == 1                    # into the pool itself
    assert g(B=0) == 0 and g(S=0) == 0


def _prefill(lib, **kw):
    a = dict(A, B=2, T=5, S=50, ks=0, H=4, N=128, P=64, V=128, mq=4, scale=0.1, dtype=1)
    a.update(kw)
    return lib.pa_latent_prefill(a["out"], a["q"], a["kv"], a["key"], a["q_start"],
                                 a["kv_start"], a["B"], a["T"], a["S"], a["ks"], a["H"], a["N"],
                                 a["P"], a["V"], a["mq"], a["scale"], a["dtype"], None, None)


def test_prefill_refusals(lib):
    def g(**kw):
        return _prefill(lib, **kw)
    assert g(N=64) == 2 and g(P=32) == 2 and g(V=64) == 2 and g(dtype=5) == 2
    assert g(B=-1) == 1 and g(T=-1) == 1 and g(S=-1) == 1 and g(H=0) == 1 and g(mq=-1) == 1
    assert g(scale=float("nan")) == 1 and g(ks=56) == 1 and g(ks=68) == 1
    for p in ("out", "q", "kv", "key", "q_start", "kv_start"):
        assert g(**{p: None}) == 1, p
    for p in ("out", "q", "kv", "key"):
        assert g(**{p: A[p] + 8}) == 1, p
    assert g(B=0) == 0 and g(T=0) == 0 and g(mq=0) == 0


def test_strides_whose_products_pass_64_bits(lib):
    far, many = 1 << 40, 1 << 30
    assert _append(lib, qh=1 << 61, qs=far) == 1 and _append(lib, oh=1 << 61, os=far) == 1
    assert _append(lib, qh=1 << 60, os=far) == 1         # the token stride is then 2^63
    for s in ("xs", "ks", "qs", "os"):
        assert _append(lib, T=many, **{s: far}) == 1, s
    assert _gather(lib, S=many, os=far) == 1


@pytest.mark.parametrize("f", [_tree, _latent], ids=["tree", "latent"])
def test_counts_of_work_that_pass_32_bits(lib, f):
    kw = dict(mask=None, T=1, mx=1 << 24)
    assert f(lib, B=1 << 30, mq=4096, **kw) == 1
    if f is _tree:                                       # 2^30 x 2^24 x 2^9: 64 bits wrap
        assert f(lib, B=1 << 30, Hq=1 << 24, H=1 << 24, mq=65536, **kw) == 1


def test_prefill_work_that_passes_64_bits(lib):
    assert _prefill(lib, B=1 << 30, T=1, S=1, H=1 << 20, mq=1 << 22) == 1
    assert _prefill(lib, B=1 << 30, T=1, S=1, H=1 << 20, mq=(1 << 31) - 1) == 1


def test_binding_refuses_what_the_library_cannot_see(lib):
    import paged_kv_cache_301_gb300 as pa
    bf = torch.bfloat16
    q, pool = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(6, 16, 2, 64, dtype=bf)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    kw = dict(max_q_len=1, max_seq_len=48, workspace=ws)
    with pytest.raises(ValueError, match="device"):                # CPU tensors
        pa.pa_decode_tree(q, q, pool, pool, t, n, None, 0.1, **kw)
    with pytest.raises(ValueError, match="pools"):
        pa.pa_decode_tree(q, q, pool.half(), pool, t, n, None, 0.1, **kw)
    with pytest.raises(ValueError, match="tree_mask"):
        pa.pa_decode_tree(q, q, pool, pool, t, n, None, 0.1, n, **kw)
    with pytest.raises(ValueError, match="q_start"):
        pa.pa_decode_tree(q[:1], q[:1], pool, pool, t, n, None, 0.1, **kw)
    lat, ql = torch.zeros(6, 16, 320, dtype=bf), torch.zeros(2, 4, 320, dtype=bf)
    ol = torch.zeros(2, 4, 256, dtype=bf)
    with pytest.raises(ValueError, match="device"):
        pa.pa_latent_decode(ol, ql, lat, t, n, 0.1, **kw)
    with pytest.raises(ValueError, match="pool"):
        pa.pa_latent_decode(ol, ql, lat[..., :300].contiguous(), t, n, 0.1, **kw)
    with pytest.raises(ValueError, match="max_seq_len"):
        pa.pa_latent_decode(ol, ql, lat, t, n, 0.1, max_q_len=1, max_seq_len=1 << 33, workspace=ws)
    x = torch.zeros(2, 320, dtype=bf)
    with pytest.raises(ValueError, match="device"):
        pa.pa_latent_append(lat, x[:, :256], x[:, 256:], None, t, n)
    with pytest.raises(ValueError, match="share"):
        pa.pa_latent_append(lat, x[:1, :256].expand(2, 256), x[:, 256:], None, t, n)
    with pytest.raises(ValueError, match="together"):
        pa.pa_latent_append(lat, x[:, :256], x[:, 256:], None, t, n, q_rope=q)
    with pytest.raises(ValueError, match="packed"):
        pa.pa_latent_append(lat, x[:, ::2][:, :128].repeat(1, 2)[:, :256].t().contiguous().t(),
                            x[:, 256:], None, t, n)
    with pytest.raises(ValueError, match="device"):
        pa.pa_latent_gather(x, lat, t, n, torch.zeros(3, dtype=torch.int32))
    kv, o = torch.zeros(5, 4, 256, dtype=bf), torch.zeros(2, 4, 128, dtype=bf)
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        pa.pa_latent_prefill(o, torch.zeros(2, 4, 192, dtype=bf), kv, torch.zeros(5, 64, dtype=bf),
                             s, s, 0.1, max_q_len=2)
    with pytest.raises(ValueError, match="kv is"):
        pa.pa_latent_prefill(o, torch.zeros(2, 4, 200, dtype=bf), kv, torch.zeros(5, 64, dtype=bf),
                             s, s, 0.1, max_q_len=2)

"""Argument checks of the rotated cache writes and the 8-bit cache: every refusal comes
back before any launch (CPU only: no kernel runs)."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_301_gb300 import build
    build.build()
    from paged_kv_cache_301_gb300 import _lib
    return _lib.load()


# addresses far apart, so that nothing overlaps; no kernel runs
A = {n: (i + 1) << 32 for i, n in enumerate(
    "q_out k_pool v_pool k_scale v_scale q key value q_weight k_weight cos_sin positions tables "
    "lens q_start out ws pairs".split())}


def _rope(lib, name, **kw):
    a = dict(A, eps=1e-6, P=64, R=128, inter=0, positions=None, q_start=None, B=4, T=4, qs=0,
             ks=0, Hq=8, H=2, D=128, bs=16, MB=4, NB=20, dtype=1)
    a.update(kw)
    scales = [a["k_scale"], a["v_scale"]] if name.endswith("q8") else []
    return getattr(lib, name)(
        a["q_out"], a["k_pool"], a["v_pool"], *scales, a["q"], a["key"], a["value"],
        a["q_weight"], a["k_weight"], a["eps"], a["cos_sin"], a["P"], a["R"], a["inter"],
        a["positions"], a["tables"], a["lens"], a["q_start"], a["B"], a["T"], a["qs"], a["ks"],
        a["Hq"], a["H"], a["D"], a["bs"], a["MB"], a["NB"], a["dtype"], None, None)


@pytest.mark.parametrize("name", ["pa_rope_append", "pa_rope_append_q8"])
def test_rope_refusals(lib, name):
    def f(**kw):
        return _rope(lib, name, **kw)
    assert f(D=96) == 2 and f(bs=12) == 2 and f(dtype=3) == 2
    assert f(B=-1) == 1 and f(T=-1) == 1 and f(Hq=0) == 1 and f(H=0) == 1
    assert f(MB=0) == 1 and f(NB=0) == 1
    assert f(R=120) == 1 and f(R=144) == 1 and f(R=-16) == 1      # rotary_dim
    assert f(P=0) == 1 and f(cos_sin=None) == 1                   # rotation without a table
    assert f(eps=float("nan")) == 1 and f(eps=-1.0) == 1 and f(eps=float("inf")) == 1
    assert f(T=5) == 1                          # no q_start: one token per sequence
    assert f(qs=8 * 128 - 8) == 1 and f(qs=8 * 128 + 4) == 1
    assert f(ks=2 * 128 - 8) == 1 and f(ks=2 * 128 + 4) == 1
    for p in ("q_out", "k_pool", "v_pool", "q", "key", "value", "tables", "lens"):
        assert f(**{p: None}) == 1, p
    for p in ("q_out", "k_pool", "v_pool", "q", "key", "value", "q_weight", "k_weight", "cos_sin"):
        assert f(**{p: A[p] + 8}) == 1, p                         # 16-byte alignment
    assert f(q_out=A["q"], qs=12 * 128) == 1    # in place needs packed rows
    assert f(q_out=A["q"] + 256) == 1           # a shifted overlap
    assert f(q_out=A["key"]) == 1 and f(q_out=A["value"] + 16) == 1
    assert f(B=0, T=0) == 0
    assert f(B=3, T=0, q_start=A["q_start"]) == 0                 # nothing to do
    if name.endswith("q8"):
        assert f(k_scale=None) == 1 and f(v_scale=None) == 1 and f(k_scale=A["k_scale"] + 2) == 1


def _decode(lib, **kw):
    a = dict(A, B=2, Hq=8, H=2, D=128, bs=16, MB=4, NB=8, mx=64, scale=0.1, dtype=1,
             ws_bytes=1 << 30)
    a.update(kw)
    return lib.pa_decode_q8(a["out"], a["q"], a["k_pool"], a["v_pool"], a["k_scale"], a["v_scale"],
                            a["tables"], a["lens"], a["B"], a["Hq"], a["H"], a["D"], a["bs"],
                            a["MB"], a["NB"], a["mx"], a["scale"], a["dtype"], a["ws"],
                            a["ws_bytes"], None, None)


def test_decode_q8_refusals(lib):
    def f(**kw):
        return _decode(lib, **kw)
    assert f(D=96) == 2 and f(bs=12) == 2 and f(dtype=5) == 2
    assert f(Hq=7) == 1 and f(B=-1) == 1 and f(mx=65) == 1 and f(mx=-1) == 1
    assert f(MB=0) == 1 and f(NB=0) == 1
    assert f(scale=float("nan")) == 1 and f(scale=float("inf")) == 1
    for p in ("out", "q", "k_pool", "v_pool", "k_scale", "v_scale", "tables", "lens"):
        assert f(**{p: None}) == 1, p
    for p in ("out", "q", "k_pool", "v_pool"):
        assert f(**{p: A[p] + 8}) == 1, p
    assert f(k_scale=A["k_scale"] + 2) == 1
    assert f(ws=None) == 3 and f(ws=A["ws"] + 16) == 3 and f(ws_bytes=0) == 3
    assert f(B=0) == 0


def test_decode_q8_workspace_query(lib):
    f = lib.pa_decode_q8_workspace_bytes
    n = f(64, 32, 8, 128, 16, 4096)
    assert n > 0 and n % 256 == 0
    assert f(64, 32, 8, 96, 16, 4096) == 0 and f(64, 32, 8, 128, 12, 4096) == 0
    assert f(64, 33, 8, 128, 16, 4096) == 0 and f(-1, 32, 8, 128, 16, 4096) == 0
    assert f(64, 32, 8, 128, 16, -1) == 0


def _expand(lib, **kw):
    a = dict(A, n=3, H=2, D=128, bs=16, sn=8, dn=8, dtype=1, k8=1 << 40, v8=1 << 41)
    a.update(kw)
    return lib.pa_expand_blocks_q8(a["k_pool"], a["v_pool"], a["k8"], a["v8"], a["k_scale"],
                                   a["v_scale"], a["pairs"], a["n"], a["H"], a["D"], a["bs"],
                                   a["sn"], a["dn"], a["dtype"], None, None)


def test_expand_refusals(lib):
    def f(**kw):
        return _expand(lib, **kw)
    assert f(D=96) == 2 and f(bs=12) == 2 and f(dtype=7) == 2
    assert f(n=-1) == 1 and f(H=0) == 1 and f(sn=0) == 1 and f(dn=0) == 1
    for p in ("k_pool", "v_pool", "k8", "v8", "k_scale", "v_scale", "pairs"):
        assert f(**{p: None}) == 1, p
    for p in ("k_pool", "v_pool"):
        assert f(**{p: A[p] + 8}) == 1, p
    assert f(k8=(1 << 40) + 8) == 1 and f(v_scale=A["v_scale"] + 1) == 1
    assert f(n=0) == 0


def test_binding_refuses_what_the_library_cannot_see(lib):
    """Shapes, dtypes and devices: checked in Python, before any address is passed on."""
    import paged_kv_cache_301_gb300 as pa
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pool8, sc = torch.zeros(6, 2, 16, 64, dtype=torch.uint8), torch.ones(6, 2)
    with pytest.raises(ValueError, match="device"):                # CPU tensors
        pa.pa_rope_append(q, torch.zeros(6, 16, 2, 64), torch.zeros(6, 16, 2, 64), q, k, k, None,
                          t, n)
    pools = torch.zeros(6, 16, 2, 64), torch.zeros(6, 16, 2, 64)
    for qkv in ((q[:1].expand(2, 4, 64), k, k), (q, *[k[:1].expand(2, 2, 64)] * 2)):
        with pytest.raises(ValueError, match="stride of 0"):       # one row for all tokens
            pa.pa_rope_append(q, *pools, *qkv, None, t, n)
    with pytest.raises(ValueError, match="packed"):
        pa.pa_rope_append(q, *pools, q[:, :1].expand(2, 4, 64), k, k, None, t, n)
    with pytest.raises(ValueError, match="device"):
        pa.pa_decode_q8(q, q, pool8, pool8, sc, sc, t, n, 0.1)
    with pytest.raises(ValueError, match="8-bit pools"):
        pa.pa_decode_q8(q, q, pool8.float(), pool8.float(), sc, sc, t, n, 0.1)
    with pytest.raises(ValueError, match="scales"):
        pa.pa_decode_q8(q, q, pool8, pool8, sc.t(), sc, t, n, 0.1)
    with pytest.raises(ValueError, match="device"):
        pa.pa_expand_blocks_q8(torch.zeros(6, 16, 2, 64), torch.zeros(6, 16, 2, 64), pool8, pool8,
                               sc, sc, t)


def test_rope_table_is_fp64_rounded_once():
    import paged_kv_cache_301_gb300 as pa
    t = pa.rope_table(100_003, 32, base=500000.0, device="cpu")
    assert t.shape == (100_003, 32) and t.dtype == torch.float32
    for p, j in ((0, 0), (7, 3), (100_002, 0), (100_002, 15)):
        a = p * 500000.0 ** (-2 * j / 32)
        assert abs(float(t[p, j]) - math.cos(a)) <= 2.0 ** -24
        assert abs(float(t[p, 16 + j]) - math.sin(a)) <= 2.0 ** -24

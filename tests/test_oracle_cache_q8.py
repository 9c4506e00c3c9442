"""Pins of the oracle's norm, rotation and 8-bit cache against things other than itself:
torch's float8 conversion, complex multiplication, closed forms (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import cache_q8 as oq


def test_e4m3_codes_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    v = oq.decode_e4m3(codes)
    assert np.array_equal(np.isnan(t), np.isnan(v))
    assert np.array_equal(t[~np.isnan(t)], v[~np.isnan(v)])
    assert v[0x7E] == 448.0 and np.isnan(v[0x7F])


def test_e4m3_rounding_matches_torch_with_ties_to_even():
    g = np.random.default_rng(0)
    mid = (oq.VALUES[:-1] + oq.VALUES[1:]) / 2
    x = np.concatenate([mid, -mid, g.normal(size=4000) * 60, g.normal(size=2000) * 0.01,
                        oq.VALUES, [0.0, -0.0]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oq.encode_e4m3(x), want)
    assert list(oq.encode_e4m3(np.array([1e9, np.inf, -np.inf, 460.0]))) == [0x7E, 0x7E, 0xFE, 0x7E]
    assert oq.encode_e4m3(np.array([np.nan]))[0] == 0x7F


def test_scale_is_the_smallest_power_of_two_that_fits():
    g = np.random.default_rng(1)
    for a in list(np.exp(g.uniform(-30, 30, 200))) + [448.0, 448.0001, 224.0, 896.0, 3.5, 7.0]:
        s = oq.scale_for(a)
        assert np.log2(s) == int(np.log2(s))
        assert a <= 448 * s and a > 448 * s / 2
    assert oq.scale_for(0.0) == 2.0 ** -64
    assert oq.scale_for(1e-30) == 2.0 ** -64


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [16, 48, 64])
def test_rotation_is_multiplication_by_a_unit_complex_number(interleaved, R):
    g = np.random.default_rng(2)
    x = g.normal(size=(5, 3, 64))
    th = g.uniform(-10, 10, size=(5, R // 2))
    y = oq.rotate(x, np.concatenate([np.cos(th), np.sin(th)], -1), interleaved)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * th)[:, None]
    assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
    assert np.array_equal(y[..., R:], x[..., R:])


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(3).normal(size=(7, 2, 128)) * 5
    y = oq.rms_norm(x, np.ones(128), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    assert oq.rms_norm(x, None, 1e-6) is x


def test_appending_one_by_one_stays_near_the_values():
    """Blocks filled token by token: each stored value is within half a code step of the
    value at the block's final scale, plus half a subnormal step for each rescale."""
    g = np.random.default_rng(4)
    bs, H, D, L = 8, 2, 64, 21
    rows = g.normal(size=(L, H, D)) * np.exp(g.normal(size=(L, 1, 1)))
    codes = np.zeros((4, H, bs, D), dtype=np.uint8)
    scales = np.ones((4, H))
    table = [[2, 0, 3]]
    for n in range(1, L + 1):
        oq.append_q8(codes, scales, rows[n - 1:n], [(0, 0, n - 1, table[0][(n - 1) // bs], (n - 1) % bs)])
    v = oq.values_q8(codes, scales)
    pos = np.arange(L)
    got = v[np.array(table[0])[pos // bs], pos % bs]
    s = scales[np.array(table[0])[pos // bs]][:, :, None]
    assert (np.abs(got - rows) <= np.abs(rows) * 2.0 ** -4 + bs * s * 2.0 ** -10).all()


def test_one_call_and_block_by_block_calls_agree():
    g = np.random.default_rng(5)
    bs, H, D = 8, 2, 64
    rows = g.normal(size=(24, H, D))
    tables = [[1, 3, 0]]
    both = []
    for cuts in ([0, 24], [0, 8, 16, 24]):
        codes, scales = np.zeros((4, H, bs, D), dtype=np.uint8), np.ones((4, H))
        for a, b in zip(cuts, cuts[1:]):
            oq.append_q8(codes, scales, rows[a:b],
                         oq.placements([b], [0, b - a], tables, bs))
        both.append((codes, scales))
    assert np.array_equal(both[0][0], both[1][0]) and np.array_equal(both[0][1], both[1][1])


def test_decode_matches_a_library_softmax():
    g = np.random.default_rng(6)
    bs, H, D, G, L = 8, 2, 64, 3, 19
    codes = g.integers(0, 0x7F, size=(6, H, bs, D)).astype(np.uint8)
    scales = 2.0 ** g.integers(-9, -5, size=(6, H))
    v = oq.values_q8(codes, scales)
    q = g.normal(size=(H * G, D))
    table = [4, 0, 5]
    out, mass, size = oq.decode_with_spread(q, v, v[::-1], table, L, 0.02)
    kk = torch.from_numpy(np.concatenate([v[i] for i in table])[:L].copy())
    vv = torch.from_numpy(np.concatenate([v[::-1][i] for i in table])[:L].copy())
    for h in range(H * G):
        p = torch.softmax(0.02 * kk[:, h // G] @ torch.from_numpy(q[h]), 0)
        assert np.allclose(out[h], (p @ vv[:, h // G]).numpy())
    assert (mass >= np.abs(out) - 1e-12).all() and (size > 0).all()
    zero = oq.decode_with_spread(q, v, v, table, 0, 0.02)[0]
    assert not zero.any()

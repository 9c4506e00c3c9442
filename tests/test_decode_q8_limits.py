"""Sizes that pa_decode_q8's 32-bit arithmetic does not hold are refused before any launch
(CPU only: no kernel runs)."""
import pytest

from tests.test_rope_q8_abi import _decode


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_301_gb300 import build
    build.build()
    from paged_kv_cache_301_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("kw", [
    # the cost of one sequence's items, 4 a tile, is taken apart in 32 bits
    dict(mx=1 << 30, H=64, Hq=64, bs=64, MB=1 << 24),            # 2^23 tiles of 64 heads
    dict(mx=1 << 30, H=1, Hq=512, bs=64, MB=1 << 24),            # of 64 chunks of one head
    dict(mx=1 << 30, H=128, Hq=128, D=64, bs=64, MB=1 << 24),    # 2^22 tiles of 128 heads
    dict(mx=(1 << 31) - 128, H=32, Hq=32, bs=64, MB=1 << 25),
    # a length rounded up to tiles, and a block's place in a tile, are ints
    dict(mx=(1 << 31) - 1, bs=64, MB=1 << 25),
    dict(mx=(1 << 31) - 2047, H=1, Hq=1, D=64, bs=64, MB=1 << 25),
    # what was refused before
    dict(mx=1 << 30, B=32, bs=64, MB=1 << 24),                   # tiles of all sequences
    dict(H=1 << 20, Hq=1 << 20),                                 # items of a sequence
    dict(NB=1 << 20, H=128, Hq=128),                             # rows of a pool
])
def test_refused(lib, kw):
    assert _decode(lib, **kw) == 1

"""PA_TWO_TERMS in a dtype: the calls that know it, what it leaves refused (CPU only: no kernel
runs)."""
from tests.test_latent_abi import _append, _gather, _latent, _prefill, _tree, lib  # noqa: F401

TWO = 0x100


def test_the_flag_is_one_of_the_attention_calls(lib):      # noqa: F811
    for f in (_tree, _latent, _prefill):
        for dtype in (0, 1):
            # known: what is refused is the argument behind it
            assert f(lib, dtype=dtype | TWO, B=-1) == 1
            assert f(lib, dtype=dtype | TWO, T=0) == 0
        for dtype in (5 | TWO, 2 * TWO, 1 | 3 * TWO, TWO | 2):
            assert f(lib, dtype=dtype) == 2, (f, dtype)
    assert _append(lib, dtype=1 | TWO) == 2 and _gather(lib, dtype=1 | TWO) == 2


def test_the_workspace_is_that_of_one_term(lib):           # noqa: F811
    for f, kw in ((_tree, dict(Hq=64, H=2)), (_latent, dict(Hq=128))):
        assert f(lib, dtype=1 | TWO, ws_bytes=0, **kw) == 3

"""Which rows share a byte (csrc/pa_share.h, by a host compiler), against sets of bytes; and the
latent write's refusals that follow from it (CPU only: no kernel runs)."""
import os
import subprocess

import numpy as np
import pytest

from tests.test_latent_abi import A, _append, lib  # noqa: F401  (lib: a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r'''
#include <cstdio>
#include "%s/paged_kv_cache_301_gb300/csrc/pa_share.h"
using namespace pa;
int main() {
  long long b[2], T, s[2], n[2], h[2], w[2];
  while (scanf("%%lld", &T) == 1) {
    Rows r[2];
    for (int i = 0; i < 2; ++i) {
      if (scanf("%%lld %%lld %%lld %%lld %%lld", &b[i], &s[i], &n[i], &h[i], &w[i]) != 5) return 1;
      r[i] = {(const void*)(uintptr_t)b[i], T, s[i], n[i], h[i], w[i]};
    }
    printf("%%d\n", (int)share(r[0], r[1]));
  }
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("share")
    src, exe = d / "s.cpp", d / "s"
    src.write_text(SOURCE % ROOT)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", str(exe), str(src)], check=True)
    return str(exe)


def bytes_of(b, T, s, n, h, w):
    return {b + t * s + i * h + k for t in range(T) for i in range(n) for k in range(w)}


def test_against_sets(program):
    g = np.random.default_rng(1)
    cases, want, told = [], [], []
    for _ in range(4000):
        T = int(g.integers(1, 4))
        rows = []
        stride = int(g.integers(40, 90))
        head = int(g.integers(5, 14))
        for i in range(2):
            n, w = int(g.integers(1, 5)), int(g.integers(2, 6))
            h = head if g.random() < 0.8 else int(g.integers(5, 14))
            h = max(h, w)
            extent = (n - 1) * h + w
            s = stride if g.random() < 0.9 else int(g.integers(40, 90))
            s = max(s, extent)
            rows.append((int(g.integers(1000, 1160)), s, n, h, w))
        cases.append(f"{T} " + " ".join(" ".join(map(str, r)) for r in rows))
        x, y = (bytes_of(b, T, s, n, h, w) for b, s, n, h, w in rows)
        want.append(bool(x & y))
        (_, s0, n0, h0, w0), (_, s1, n1, h1, w1) = rows
        # exact for one stride and one distance of heads, behind the first and last token too
        told.append((T == 1 or s0 == s1) and (n0 == 1 or n1 == 1 or (h0 == h1 and w0 == w1)))
    out = subprocess.run([program], input="\n".join(cases) + "\n", capture_output=True, text=True,
                         check=True).stdout.split()
    got = [x == "1" for x in out]
    assert len(got) == len(want)
    wrong = [c for c, a, b in zip(cases, got, want) if b and not a]
    assert not wrong, wrong[:3]                            # no shared byte is missed
    exact = [(c, a, b) for c, a, b, t in zip(cases, got, want, told) if t and c[0] == "1"]
    assert len(exact) > 500 and all(a == b for _, a, b in exact)
    same = [(a, b) for a, b, t in zip(got, want, told) if t]
    assert sum(a != b for a, b in same) < len(same) // 20  # only ends of the rows


def test_append_refuses_shared_bytes(lib):                 # noqa: F811
    def g(**kw):
        return _append(lib, **kw)
    q = A["q_rope"]
    # [q heads | latent | key] of one projection: 8 heads of 64, 512, 64; out 16 bytes into each
    wide = dict(latent=q + 2 * 512, key=q + 2 * 1024, qs=1088, xs=1088, ks=1088, os=1088)
    assert g(**wide, q_out=q + 2 * 448, Hq=8) == 1         # its last head in the latent part
    assert g(**wide, q_out=q + 2 * 1024, Hq=1) == 1        # the key part itself
    assert g(**wide, q_out=q + 2 * 8, Hq=8) == 1           # shifted within the heads
    assert g(q_out=q + 2 * 32, Hq=1, qs=128, os=128) == 1  # one head, half of it
    assert g(q_out=q + 2 * 96, Hq=1, qs=128, os=128) == 1  # into the next token's head
    assert g(q_out=q, Hq=1, qs=128, os=192) == 1           # in place with other token strides
    assert g(q_out=q, Hq=2, qs=256, os=256, oh=128) == 1   # or other head strides


def test_append_refuses_inputs_that_it_writes(lib):        # noqa: F811
    def g(**kw):
        return _append(lib, **kw)
    inside = A["pool"] + 64                                # 8 blocks of 16 rows of 1,152 bytes
    last = A["pool"] + 8 * 16 * 1152 - 16
    none = dict(q_rope=None, q_out=None)
    for p in ("latent", "key", "weight", "cos_sin", "positions", "tables", "lens", "q_start"):
        for at in (inside, last):
            assert g(**{p: at}) == 1 and g(**none, **{p: at}) == 1, p
    assert g(q_rope=inside) == 1 and g(q_out=last) == 1
    assert g(latent=A["pool"] - 1024) == 1                 # its fifth row's end is in the pool
    for p in ("weight", "cos_sin", "tables", "lens", "q_start"):
        assert g(q_out=A[p]) == 1, p
    assert g(positions=A["q_out"] + 64) == 1
    assert g(q_out=A["weight"] + 2 * 512 - 16) == 1        # its last bytes
    assert g(q_out=A["cos_sin"] + 64 * 64 * 4 - 16) == 1
    assert g(B=(1 << 31) - 1, MB=(1 << 31) - 1) == 1       # tables of 2^64 bytes: all of memory

"""How the attention of several new tokens cuts its work into windows, from the kernel's own
header and a host compiler (CPU only): against a walk over all tiles."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r'''
#include <cstdio>
#include <vector>
#include "%s/paged_kv_cache_301_gb300/csrc/pa_multi_window.cuh"
using namespace pa::multi;
// B, sets, ends, threads, then nt and items of each sequence; prints each window's place
template <class I>
void run(int B, int sets, int ends, int threads, const std::vector<Work>& w) {
  I tiles = 0, items = 0;
  for (auto& x : w) { tiles += (I)x.nt * x.items; items += x.nt ? x.items : 0; }
  auto work_of = [&](int b) { return w[b]; };
  const Cut<I> cut = cut_of<I>(tiles, items, sets, ends);
  printf("cut %%lld %%lld %%d %%d\n", (long long)cut.tiles, (long long)cut.total, cut.windows, cut.ends);
  const int per = (B + threads - 1) / threads;
  for (int c = 0; c < cut.windows; ++c) {
    const I at = bound_of(cut, c);
    int found = 0;
    I t = 0, n = 0;
    for (int i = 0; i < threads; ++i) {
      Share<I> s;
      s.b0 = i * per < B ? i * per : B;
      s.b1 = s.b0 + per < B ? s.b0 + per : B;
      s.tiles_to = t; s.items_to = n; s.tiles = s.items = 0;
      for (int b = s.b0; b < s.b1; ++b) {
        s.tiles += (I)w[b].nt * w[b].items;
        s.items += w[b].nt ? w[b].items : 0;
      }
      t += s.tiles; n += s.items;
      Place<I> p;
      if (place_of(cut, s, B, at, work_of, &p)) {
        ++found;
        printf("%%d %%lld %%d %%d %%d\n", c, (long long)p.lin, p.b, p.item, p.j);
      }
    }
    if (found != 1) { printf("found %%d\n", found); return; }
  }
}
int main() {
  int B, sets, ends, threads, wide;
  while (scanf("%%d %%d %%d %%d %%d", &B, &sets, &ends, &threads, &wide) == 5) {
    std::vector<Work> w(B);
    for (auto& x : w) if (scanf("%%d %%d", &x.nt, &x.items) != 2) return 1;
    if (wide) run<int64_t>(B, sets, ends, threads, w); else run<int>(B, sets, ends, threads, w);
    printf("end\n");
  }
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("windows")
    src, exe = d / "w.cpp", d / "w"
    src.write_text(SOURCE % ROOT)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", str(exe), str(src)], check=True)
    return str(exe)


def _ask(program, B, sets, ends, threads, wide, nt, items):
    text = f"{B} {sets} {ends} {threads} {wide}\n" + "".join(f"{a} {b}\n" for a, b in zip(nt, items))
    out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout
    lines = [x.split() for x in out.strip().splitlines()]
    assert lines[-1] == ["end"]
    assert lines[0][0] == "cut"
    return [int(x) for x in lines[0][1:]], [[int(x) for x in ln] for ln in lines[1:-1]]


@pytest.mark.parametrize("seed", range(40))
def test_windows_cover_every_tile_once(program, seed):
    g = np.random.default_rng(seed)
    B = int(g.integers(1, 40)) if seed % 3 else int(g.integers(300, 900))
    nt = g.integers(0, [2, 5, 40, 3000][seed % 4], size=B)
    items = np.where(nt > 0, g.integers(1, [2, 9, 70][seed % 3], size=B), 0)
    sets = int(g.choice([1, 2, 76, 152]))
    ends = int(g.choice([0, 4, 8, 12]))
    row = [(b, i, j) for b in range(B) for i in range(items[b]) for j in range(nt[b])]
    if not row:
        return
    cut, at = _ask(program, B, sets, ends, int(g.choice([224, 352])), seed % 2, nt, items)
    assert cut[0] == len(row) and cut[2] == min(sets, len(row))
    assert len(at) == cut[2]
    lin = [a[1] for a in at]
    assert lin[0] == 0 and all(x < y for x, y in zip(lin, lin[1:])) and lin[-1] < len(row)
    for _, n, b, i, j in at:
        assert row[n] == (b, i, j)
    # equal shares: a window costs at most one tile's begin more than the average
    cost, e = 0, cut[3]
    begins = []
    for b, i, j in row:
        begins.append(cost)
        cost += 4 + (e if j == 0 else 0)
    spans = [begins[y] - begins[x] for x, y in zip(lin, lin[1:])]
    assert all(s <= cut[1] / cut[2] + 4 + e + 1 for s in spans)


def test_costs_past_32_bits(program):
    nt, items = [1 << 22, 5, 1 << 22], [300, 3, 300]
    cut, at = _ask(program, 3, 152, 12, 224, 1, nt, items)
    assert cut[0] == 2 * 300 * (1 << 22) + 15 and len(at) == 152
    for _, n, b, i, j in at:
        before = sum(nt[k] * items[k] for k in range(b))
        assert n == before + i * nt[b] + j and j < nt[b] and i < items[b]

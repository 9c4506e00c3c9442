"""The 8-bit decode's cut of a batch into windows, and the join's way back from the cut to
the parts of an item: the kernels' own arithmetic (csrc/pa_q8_window.cuh), compiled for the
host and run for every CTA and thread, against a walk over the batch."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "pa_q8_window.cuh"
#include <vector>
using namespace pa;

template <int TOKENS>
int cut_all(const int* lens, int B, int items, int grid, int ends, int threads, Window* info) {
  auto len_of = [&](int b) { return lens[b]; };
  const int per = (B + threads - 1) / threads;
  std::vector<Share> share;
  int all_tiles = 0, all_seqs = 0;
  for (int t = 0; t < threads; ++t) {
    Share s = {};
    s.b0 = t * per < B ? t * per : B;
    s.b1 = s.b0 + per < B ? s.b0 + per : B;
    s.tiles_to = all_tiles;
    s.seqs_to = all_seqs;
    for (int b = s.b0; b < s.b1; ++b) {
      const int nt = (lens[b] + TOKENS - 1) / TOKENS;
      s.tiles += nt;
      s.seqs += nt > 0;
    }
    all_tiles += s.tiles;
    all_seqs += s.seqs;
    share.push_back(s);
  }
  const Cut cut = cut_of(all_tiles, all_seqs, items, grid, ends);
  int wrong = 0;
  for (int c = 0; c < grid; ++c) {
    info[c] = Window{0, 0, 0, 0, 0, cut.total};
    if (c >= cut.ctas) continue;
    TilePlace first = {}, end = {}, p;
    int firsts = 0, ends_found = 0;
    if (cut.ctas == cut.work) {
      for (const Share& s : share)
        if (place_of_tile<TOKENS>(s, items, c, len_of, &p)) {
          first = p;
          ++firsts;
        }
      end.lin = first.lin + 1;
      ends_found = 1;
    } else {
      const Bound w0 = bound_of(cut, items, c), w1 = bound_of(cut, items, c + 1);
      for (const Share& s : share) {
        if (place_of_cost<TOKENS>(cut, s, B, items, w0, true, len_of, &p)) {
          first = p;
          ++firsts;
        }
        if (w1.at != cut.total && place_of_cost<TOKENS>(cut, s, B, items, w1, false, len_of, &p)) {
          end = p;
          ++ends_found;
        }
      }
      if (w1.at == cut.total) {
        end.lin = cut.work;
        ++ends_found;
      }
    }
    wrong += firsts != 1 || ends_found != 1;
    if (first.b < B && first.len != lens[first.b]) ++wrong;
    info[c] = Window{first.b, first.item, first.j, (int)(end.lin - first.lin), first.final,
                     cut.total};
  }
  return wrong;
}

extern "C" int cut_batch(const int* lens, int B, int tokens, int items, int grid, int ends,
                         int threads, Window* info) {
  return tokens == 128 ? cut_all<128>(lens, B, items, grid, ends, threads, info)
                       : cut_all<256>(lens, B, items, grid, ends, threads, info);
}
// The parts that the CTA of boundary c joins, their number (0: none).
extern "C" int parts_of(const Window* info, int grid, int c, int64_t* rows) {
  bool same;
  if (!first_cut(info[c], info[c - 1], &same)) return 0;
  const int n = last_window(info[c], grid) - c + 2;
  for (int k = 0; k < n; ++k) rows[k] = part_of_item(c, same, k);
  return n;
}
"""
WINDOW = np.dtype([("b", "i4"), ("item", "i4"), ("j", "i4"), ("tiles", "i4"), ("final", "i8"),
                   ("total", "i8")])


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("windows")
    (d / "windows.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "paged_kv_cache_301_gb300", "csrc")
    subprocess.run(["g++", "-x", "c++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I" + csrc,
                    "-o", str(d / "windows.so"), str(d / "windows.cpp")], check=True)
    return ctypes.CDLL(str(d / "windows.so"))


def check(lib, lens, tokens, items, grid, ends, threads=224):
    lens = np.ascontiguousarray(lens, dtype=np.int32)
    info = np.zeros(grid, dtype=WINDOW)
    wrong = lib.cut_batch(ctypes.c_void_p(lens.ctypes.data), len(lens), tokens, items, grid, ends,
                          threads, ctypes.c_void_p(info.ctypes.data))
    assert wrong == 0                      # one thread finds each end of each window
    nt = [-(-int(n) // tokens) for n in lens]
    live = [b for b, n in enumerate(nt) if n]
    work = sum(nt) * items
    at, whole, cut = [0, 0, 0], set(), {}  # place in `live`, item, tile
    for c in range(grid):
        left = int(info["tiles"][c])
        assert (left > 0) == (c < min(work, grid))
        if left:
            assert (info["b"][c], info["item"][c], info["j"][c]) == (live[at[0]], at[1], at[2])
        segment = 0
        while left:
            b = live[at[0]]
            n = min(nt[b] - at[2], left)
            if n == nt[b]:
                whole.add((b, at[1]))
            else:
                cut.setdefault((b, at[1]), []).append(2 * c + (segment > 0))
            segment, left, at[2] = segment + 1, left - n, at[2] + n
            if at[2] == nt[b]:
                at[1], at[2] = at[1] + 1, 0
                if at[1] == items:
                    at[0], at[1] = at[0] + 1, 0
    assert at == [len(live), 0, 0]         # every tile is in a window
    rows, joined = (ctypes.c_int64 * (grid + 2))(), {}
    for c in range(1, grid):
        n = lib.parts_of(ctypes.c_void_p(info.ctypes.data), grid, c, rows)
        if n:
            item = (int(info["b"][c]), int(info["item"][c]))
            assert item not in joined and n <= grid
            joined[item] = list(rows[:n])
    assert joined == cut                   # the parts that were left, in order, once
    assert not whole & set(cut)


ENDS = [0, 1, 2, 4]


@pytest.mark.parametrize("ends", ENDS)
@pytest.mark.parametrize("tokens", [128, 256])
def test_random_batches(lib, tokens, ends):
    g = np.random.default_rng(tokens + ends)
    for _ in range(400):
        B = int(g.choice([1, 2, 3, 10, 40, 100]))
        kind = g.integers(0, 6, size=B)
        lens = np.select([kind == 0, kind == 1, kind == 2, kind == 3, kind == 4],
                         [0, 1, tokens, tokens + 1, g.integers(0, 3000, size=B)],
                         g.integers(0, 40000, size=B))
        check(lib, lens, tokens, int(g.choice([1, 2, 3, 8])), int(g.choice([1, 2, 3, 7, 50, 304])),
              ends)


@pytest.mark.parametrize("ends", ENDS)
def test_more_sequences_than_threads(lib, ends):
    g = np.random.default_rng(ends)
    for B, hi in ((225, 2000), (700, 300), (3000, 600), (2048, 1024)):
        check(lib, g.integers(0, hi, size=B) * (g.integers(0, 4, size=B) > 0), 128, 8, 304, ends)
        check(lib, g.integers(0, hi, size=B), 256, 3, 160, ends)


@pytest.mark.parametrize("ends", ENDS)
def test_one_item_long_ones_and_none(lib, ends):
    for n in (1, 128, 129, 40_000, 131_072, 5_000_000):
        check(lib, [n], 128, 1, 304, ends)
        check(lib, [0, n, 0], 256, 8, 304, ends)
    check(lib, [0, 0, 0], 128, 4, 304, ends)
    check(lib, [1] * 304, 128, 1, 304, ends)
    check(lib, [1] * 305, 128, 1, 304, ends)


@pytest.mark.parametrize("ends", ENDS)
def test_costs_near_the_ends_of_32_bits(lib, ends):
    """The largest batches that the host admits: tiles times sequences below 2^28, the cost of
    one sequence's items below 2^31."""
    check(lib, [(1 << 22) * 128 - 7], 128, 127, 304, ends)         # 4 (2^22 + 1) 127 < 2^31
    check(lib, [5, (1 << 23) * 128 - 200, 9], 128, 63, 304, ends)
    check(lib, [(1 << 24) * 128 - 2048], 128, 31, 304, ends)       # the longest sequence
    check(lib, [(1 << 20) * 128] * 255, 128, 2, 304, ends)         # 2^28 - 2^20 tiles
    total = (1 << 22) // 4
    for tiles in (total - 1, total, total + 1):                    # where 64-bit division begins
        check(lib, [tiles * 128 // 8] * 8, 128, 1, 304, ends)

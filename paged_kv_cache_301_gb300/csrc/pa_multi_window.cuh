// How the attention of several new tokens per sequence (pa_multi.cuh) shares out its tiles:
// windows of equal cost, one to a set of CTAs, cut out of the row of all items.  Plain
// arithmetic, the same for the kernel and a host compiler.
//
// Sequence b has items_b items of nt_b tiles each (none where nt_b is 0); they stand in a row,
// sequence after sequence.  An item costs 4 for a tile and `ends` for its beginning and end:
// tile 0 begins at the item's cost 0, tile j > 0 at 4 j + ends.  Window c holds the tiles that
// begin in [total c / windows, total (c + 1) / windows).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_MULTI_HD __host__ __device__ __forceinline__
#else
#define PA_MULTI_HD inline
#endif

namespace pa {
namespace multi {

// Tiles of an item of a sequence, and its items.
struct Work {
  int nt, items;
};

struct Cut {
  int64_t tiles, total;        // of all items: tiles, cost
  int windows, ends;           // windows that hold any; what an item's ends cost
};

PA_MULTI_HD Cut cut_of(int64_t tiles, int64_t items, int sets, int ends) {
  Cut c;
  c.tiles = tiles;
  c.windows = tiles < sets ? (int)tiles : sets;
  // two tiles begin 4 + ends apart at most: the ends count only where windows are longer, so
  // that every window holds a tile
  c.ends = ends;
  c.total = 4 * tiles + ends * items;
  if (c.total < (int64_t)c.windows * (4 + ends)) {
    c.ends = 0;
    c.total = 4 * tiles;
  }
  return c;
}

PA_MULTI_HD int64_t bound_of(const Cut& c, int window) {
  return c.total / c.windows * window + c.total % c.windows * window / c.windows;
}

// Sequences [b0, b1) and what stands before them: tiles and items.
struct Share {
  int b0, b1;
  int64_t tiles_to, items_to, tiles, items;
};

// A window's first tile: its number among all, sequence, item of it, tile of that.
struct Place {
  int64_t lin;
  int b, item, j;
};

// The first tile that begins at cost w or behind it, if w (< total) lies in this share.
// work_of(b): sequence b's; B sequences in all.
template <class F>
PA_MULTI_HD bool place_of(const Cut& cut, const Share& s, int B, int64_t w, const F& work_of,
                          Place* p) {
  int64_t cost = 4 * s.tiles_to + cut.ends * s.items_to;
  if (w < cost || w >= cost + 4 * s.tiles + cut.ends * s.items) return false;
  int64_t tiles = s.tiles_to;
  int b = s.b0;
  Work k = work_of(b);
  for (;;) {
    const int64_t c = k.nt ? (int64_t)k.items * (4 * (int64_t)k.nt + cut.ends) : 0;
    if (w < cost + c || b + 1 >= s.b1) break;
    cost += c;
    tiles += k.nt ? (int64_t)k.items * k.nt : 0;
    k = work_of(++b);
  }
  const int64_t at = w - cost, each = 4 * (int64_t)k.nt + cut.ends;
  // 64-bit division is slow; most batches fit 32 bits
  int item = at < (1ll << 32) && each < (1ll << 32) ? (int)((uint32_t)at / (uint32_t)each)
                                                   : (int)(at / each);
  const int64_t r = at - item * each, up = (r - cut.ends + 3) >> 2;
  int64_t j = r == 0 ? 0 : (up > 1 ? up : 1);
  p->lin = tiles + (int64_t)item * k.nt + j;
  if (j >= k.nt) {                             // the next item, maybe of a later sequence
    j = 0;
    if (++item == k.items) {
      item = 0;
      do {
        k = ++b < B ? work_of(b) : Work{0, 0};
      } while ((k.nt == 0 || k.items == 0) && b < B);
    }
  }
  p->b = b;
  p->item = item;
  p->j = (int)j;
  return true;
}

// Where a set's window begins, for those who join what window boundaries cut.
struct alignas(16) Window {
  int b, item, j, tiles;
};

// Does the boundary where window `at` begins, `before` being the one before it, cut an item
// for the first time?  *same: `before` begins in that item too.
PA_MULTI_HD bool first_cut(const Window& at, const Window& before, bool* same) {
  *same = before.b == at.b && before.item == at.item;
  return at.tiles > 0 && at.j > 0 && !(*same && before.j > 0);
}

}  // namespace multi
}  // namespace pa

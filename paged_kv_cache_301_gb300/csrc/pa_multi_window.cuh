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

// Costs and tile numbers are of type I: int, or int64_t where they do not fit.
template <class I>
struct Cut {
  I tiles, total;              // of all items: tiles, cost
  int windows, ends;           // windows that hold any; what an item's ends cost
};

template <class I>
PA_MULTI_HD Cut<I> cut_of(I tiles, I items, int sets, int ends) {
  Cut<I> c;
  c.tiles = tiles;
  c.windows = tiles < sets ? (int)tiles : sets;
  // two tiles begin 4 + ends apart at most: the ends count only where windows are longer, so
  // that every window holds a tile
  c.ends = ends;
  c.total = 4 * tiles + ends * items;
  if (c.total < (I)c.windows * (4 + ends)) {
    c.ends = 0;
    c.total = 4 * tiles;
  }
  return c;
}

// total * window / windows, without the product that might not fit.
template <class I>
PA_MULTI_HD I bound_of(const Cut<I>& c, int window) {
  const I each = c.total / c.windows;
  return each * window + (int)(c.total - each * c.windows) * window / c.windows;
}

// Sequences [b0, b1) and what stands before them: tiles and items.
template <class I>
struct Share {
  int b0, b1;
  I tiles_to, items_to, tiles, items;
};

// A window's first tile: its number among all, sequence, item of it, tile of that.
template <class I>
struct Place {
  I lin;
  int b, item, j;
};

// The first tile that begins at cost w or behind it, if w (< total) lies in this share.
// work_of(b): sequence b's; B sequences in all.
template <class I, class F>
PA_MULTI_HD bool place_of(const Cut<I>& cut, const Share<I>& s, int B, I w, const F& work_of,
                          Place<I>* p) {
  I cost = 4 * s.tiles_to + cut.ends * s.items_to;
  if (w < cost || w >= cost + 4 * s.tiles + cut.ends * s.items) return false;
  I tiles = s.tiles_to;
  int b = s.b0;
  Work k = work_of(b);
  for (;;) {
    const I c = k.nt ? (I)k.items * (4 * (I)k.nt + cut.ends) : 0;
    if (w < cost + c || b + 1 >= s.b1) break;
    cost += c;
    tiles += k.nt ? (I)k.items * k.nt : 0;
    k = work_of(++b);
  }
  const I at = w - cost, each = 4 * (I)k.nt + cut.ends;
  int item = (int)(at / each);
  const I r = at - item * each, up = (r - cut.ends + 3) >> 2;
  I j = r == 0 ? 0 : (up > 1 ? up : 1);
  p->lin = tiles + (I)item * k.nt + j;
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

// How pa_decode_q8 shares out its tiles: windows of equal cost, one per CTA, and which parts
// of an item that window boundaries cut are joined.  Plain arithmetic, the same for the
// decode kernel that cuts, the join kernel that finds the parts again, and a host compiler.
//
// Items (KV head, head chunk) of sequence 0, then of sequence 1, and so on, each of nt tiles;
// an item costs 4 for a tile and `ends_cost` for its beginning and end.  Tile 0 of an item
// begins at cost 0, tile j > 0 at 4 j + ends_cost.  Window c holds the tiles that begin in
// [total c / ctas, total (c + 1) / ctas).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

// Where a CTA's window begins: sequence, item of it, tile; tiles in the window; where
// that item's final tile begins; the cost of all items (both in units of cost).
struct alignas(16) Window {
  int b, item, j, tiles;
  int64_t final, total;
};

// The whole cut: tiles of all items, windows that hold any, cost of all items.
struct Cut {
  int64_t work, ctas, total;
  int ends_cost;
};

PA_HD Cut cut_of(int all_tiles, int all_seqs, int items, int grid, int ends_cost) {
  Cut c;
  c.work = (int64_t)all_tiles * items;
  c.ctas = c.work < (int64_t)grid ? c.work : (int64_t)grid;
  // every window holds a tile: the cost of an item's ends counts only where windows are
  // longer than it
  c.ends_cost = ends_cost;
  c.total = (4 * (int64_t)all_tiles + ends_cost * all_seqs) * items;
  if (c.total < c.ctas * 2 * (4 + ends_cost)) {
    c.ends_cost = 0;
    c.total = 4 * c.work;
  }
  return c;
}

// Sequences [b0, b1) of a batch of B, and what stands before them: tiles (of one item of
// each sequence) and sequences that have any.
struct Share {
  int b0, b1, tiles, seqs, tiles_to, seqs_to;
};

// A place in the row of all tiles: its number, sequence, item, tile of it, the sequence's
// length, and where its item's final tile begins.
struct TilePlace {
  int64_t lin, final;
  int b, item, j, len;
};

// Where every window is one tile: the place of tile w, if it is one of this share's.
// len_of(b): the length of sequence b.
template <int TOKENS, class Len>
PA_HD bool place_of_tile(const Share& s, int items, int w, const Len& len_of, TilePlace* p) {
  const int t = w / items;
  if (t < s.tiles_to || t >= s.tiles_to + s.tiles) return false;
  int b = s.b0, tile = s.tiles_to, len = 0, nt = 0;
  for (;; ++b) {
    len = len_of(b);
    nt = (len + TOKENS - 1) / TOKENS;
    if (t < tile + nt) break;
    tile += nt;
  }
  const int at = w - tile * items, item = at / nt;
  p->b = b;
  p->item = item;
  p->j = at - item * nt;
  p->len = len;
  p->lin = w;
  p->final = 4 * (int64_t)(tile * items + item * nt + nt - 1);
  return true;
}

// The cost at which window c begins, and that divided by items (where it lies among one
// item of each sequence).
struct Bound {
  int64_t at;
  int one;
};

PA_HD Bound bound_of(const Cut& cut, int items, uint32_t c) {
  // 64-bit division takes half a microsecond; most batches fit 32 bits
  const bool narrow = cut.total < (1 << 22);
  Bound w;
  w.at = narrow ? (int64_t)((uint32_t)cut.total * c / (uint32_t)cut.ctas)
                : cut.total * c / cut.ctas;
  w.one = narrow ? (int)((uint32_t)w.at / (uint32_t)items) : (int)(w.at / items);
  return w;
}

// The first tile that begins at w or behind it, if w lies in this share; `whole`: its whole
// place, not only its number.
template <int TOKENS, class Len>
PA_HD bool place_of_cost(const Cut& cut, const Share& s, int B, int items, const Bound& w,
                         bool whole, const Len& len_of, TilePlace* p) {
  const int before = 4 * s.tiles_to + cut.ends_cost * s.seqs_to;      // of one item of each
  const int mine = 4 * s.tiles + cut.ends_cost * s.seqs;
  if (w.one < before || w.one >= before + mine) return false;
  int b = s.b0, cost = before, tile = s.tiles_to, nt = 0, len = 0;
  for (;; ++b) {
    len = len_of(b);
    nt = (len + TOKENS - 1) / TOKENS;
    const int c = nt ? 4 * nt + cut.ends_cost : 0;
    if (w.one < cost + c || b + 1 >= s.b1) break;
    cost += c;
    tile += nt;
  }
  const int c = 4 * nt + cut.ends_cost;
  const int at = (int)(w.at - (int64_t)cost * items);
  int item = at / c;
  const int r = at - item * c, up = (r - cut.ends_cost + 3) >> 2;
  int j = r == 0 ? 0 : (up > 1 ? up : 1);
  p->lin = (int64_t)tile * items + (int64_t)item * nt + j;
  if (!whole) return true;
  int64_t base = (int64_t)cost * items + (int64_t)item * c;
  if (j >= nt) {                               // the next item, maybe of a later sequence
    j = 0;
    base += c;
    if (++item == items) {
      item = 0;
      do {
        len = ++b < B ? len_of(b) : 0;
        nt = (len + TOKENS - 1) / TOKENS;
      } while (nt == 0 && b < B);
    }
  }
  p->b = b;
  p->item = item;
  p->j = j;
  p->len = len;
  p->final = base + (nt > 1 ? 4 * (nt - 1) + cut.ends_cost : 0);
  return true;
}

// Does the boundary where window `at` begins, `before` being the one before it, cut an item
// for the first time?  *same: `before` begins in that item too.
PA_HD bool first_cut(const Window& at, const Window& before, bool* same) {
  *same = before.b == at.b && before.item == at.item;
  // not an empty window, not a boundary between items, no earlier boundary in this item
  return at.tiles > 0 && at.j > 0 && !(*same && before.j > 0);
}

// The window that holds the final tile of the item that window `at` begins in.
PA_HD int last_window(const Window& at, int grid) {
  const int64_t windows = at.total / 4 < grid ? at.total / 4 : grid;   // fewer: of a tile each
  const int64_t c = ((at.final + 1) * windows - 1) / at.total;
  return (int)(c < windows - 1 ? c : windows - 1);
}

// A window leaves two parts at most: of its first segment and of a later one (its last).
// Part k of the item that boundary c cuts first: the segment of window c - 1 that ends there,
// then the first segments of windows c, c + 1 and so on.
PA_HD int64_t part_of_item(int c, bool same, int k) {
  return 2 * (int64_t)(c - 1 + k) + (k == 0 && !same ? 1 : 0);
}

}  // namespace pa

// Whether two sets of token rows, each a few pieces of every row, share a byte: what a call that
// writes one and reads the other may be given.  Plain arithmetic on addresses.
#pragma once

#include <stdint.h>

namespace pa {

// Bytes [p, p + n) and [q, q + m).
inline bool overlaps(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t x = (uintptr_t)p, y = (uintptr_t)q;
  return x < y + (uint64_t)m && y < x + (uint64_t)n;
}

// Rows of T tokens, `stride` bytes apart: `heads` pieces of `width` bytes, `head` apart.
struct Rows {
  const void* base;
  int64_t T, stride, heads, head, width;
  int64_t extent() const { return (heads - 1) * head + width; }
  int64_t span() const { return (T - 1) * stride + extent(); }
};

// From sizes in 16-bit elements.
inline Rows rows_of(const void* p, int64_t T, int64_t stride, int64_t heads, int64_t head,
                    int64_t width) {
  return {p, T, 2 * stride, heads, 2 * head, 2 * width};
}

// Do pieces of one token's x and y, whose first piece stands d bytes behind x's, share a byte?
// Pieces at two different distances are taken to, where the tokens' extents meet.
inline bool meet(const Rows& x, const Rows& y, int64_t d) {
  if (d >= x.extent() || d + y.extent() <= 0) return false;
  if (x.heads == 1 && y.heads == 1) return true;
  if (x.heads == 1) {                          // the first piece of y that ends behind x's start
    const int64_t j = d + y.width > 0 ? 0 : (-d - y.width) / y.head + 1;
    return j < y.heads && d + j * y.head < x.width;
  }
  if (y.heads == 1) return meet(y, x, -d);
  if (x.head != y.head) return true;
  const int64_t r = (d % x.head + x.head) % x.head;
  return r < x.width || x.head - r < y.width;
}

// Do x and y share a byte?  Each token's pieces lie within its stride; rows at two different
// strides are taken to, where their spans meet.
inline bool share(const Rows& x, const Rows& y) {
  if (!overlaps(x.base, x.span(), y.base, y.span())) return false;
  const int64_t d = (intptr_t)y.base - (intptr_t)x.base;
  if (x.T == 1) return meet(x, y, d);
  if (x.stride != y.stride) return true;
  const int64_t r = (d % x.stride + x.stride) % x.stride;
  return meet(x, y, r) || meet(x, y, r - x.stride);
}

}  // namespace pa

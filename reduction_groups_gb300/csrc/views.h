// Overlap of strided row views.
#pragma once

#include <stdint.h>

namespace psk {

// Rows of `row` bytes, `stride` bytes apart, from address p (rows, row >= 1).
struct View {
  uintptr_t p;
  int64_t rows;
  uint64_t row, stride;
  uint64_t bytes() const { return (uint64_t)(rows - 1) * stride + row; }
};

inline View view_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return View{(uintptr_t)p, rows, (uint64_t)(cols * size), (uint64_t)(rows > 1 ? ld * size : cols * size)};
}

// Whether two views may share a byte.  Views with one stride (columns of one
// buffer) are compared within it; others by the range from first to last byte.
inline bool views_overlap(const View& a, const View& b) {
  if (a.rows < 1 || b.rows < 1 || a.row < 1 || b.row < 1) return false;
  if (a.p >= b.p + b.bytes() || b.p >= a.p + a.bytes()) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
    const uint64_t s = a.stride;
    const uint64_t d = (uint64_t)(b.p >= a.p ? (b.p - a.p) % s : (s - (a.p - b.p) % s) % s);   // b's start after a's
    return d < a.row || d + b.row > s;
  }
  return true;
}

inline bool same_view(const View& a, const View& b) {
  return a.p == b.p && a.rows == b.rows && a.row == b.row && a.stride == b.stride;
}

}  // namespace psk

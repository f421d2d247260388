// Whether tensors of a call share memory.  Plain C++, so that a host compiler
// can build it alone.
#pragma once

#include <stdint.h>

namespace moe {

// Rows of `width` bytes, `stride` apart (one row, or as many on the same bytes: any stride).
struct Rows {
  const void* p;
  int64_t rows, stride, width;
};
inline Rows bytes_at(const void* p, int64_t n) { return Rows{p, 1, n, n}; }

// Whether rows `a` reach into the bytes of `b`, one row: what lies between two rows of `a` is apart from them.  NULL shares nothing.
inline bool rows_meet(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.rows <= 0 || a.width <= 0 || b.rows <= 0 || b.width <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p), b1 = b0 + (uintptr_t)b.width;
  const int64_t rows = a.stride > 0 ? a.rows : 1;
  if (a0 >= b1 || b0 >= a0 + (uintptr_t)((rows - 1) * a.stride + a.width)) return false;
  if (rows == 1 || b0 < a0 + (uintptr_t)a.width) return true;
  // the first row that ends behind b's first byte
  const uintptr_t r = (b0 - a0 - (uintptr_t)a.width) / (uintptr_t)a.stride + 1;
  return a0 + r * (uintptr_t)a.stride < b1;
}

}  // namespace moe

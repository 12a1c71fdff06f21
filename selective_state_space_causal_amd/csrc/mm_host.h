// Host helpers shared by the argument checks of every entry point.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace mm {

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && a0 < b0 + nb && b0 < a0 + na;
}

struct Span {
  const void* p;
  size_t n;
};

// `rows` rows of `n` bytes, `stride` bytes apart (contiguous arrays: one row)
struct Rows {
  const void* p;
  int64_t rows;
  size_t n;
  size_t stride;
  size_t extent() const { return rows > 0 && n > 0 ? static_cast<size_t>(rows - 1) * stride + n : 0; }
};
// Whether two such arrays share a byte.  Column ranges of one array (the same stride) are taken apart
// by where their rows lie in the stride; other strides are judged by their extents.
inline bool overlap(const Rows& a, const Rows& b) {
  if (!overlap(a.p, a.extent(), b.p, b.extent())) return false;
  if (a.stride != b.stride || a.rows <= 1 || b.rows <= 1) return true;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const size_t at = b0 >= a0 ? (b0 - a0) % a.stride : (a.stride - (a0 - b0) % a.stride) % a.stride;
  return at < a.n || at + b.n > a.stride;
}

}  // namespace mm

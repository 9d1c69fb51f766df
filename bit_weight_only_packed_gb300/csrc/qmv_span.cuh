// qmv_span.cuh -- what the host checks of a call's pointers: their alignment, and whether two
// of them share memory.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace qmv {
namespace span_of {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The bytes that a call reads or writes at one pointer: rows of `width`, `ld` apart.
struct Span {
  const void* p;
  int64_t rows, ld, width;
};
inline Span span(const void* p, int64_t rows, int64_t ld, int64_t cols, size_t size) {
  return {p, rows, ld * (int64_t)size, cols * (int64_t)size};
}
inline Span flat(const void* p, int64_t n, size_t size) { return span(p, 1, n, n, size); }

// Whether two spans share a byte.  Rows of one stride may lie between each other's
// (two halves of a wider tensor); ranges that cross with different strides are taken
// to share one.
inline bool meet(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const Span &lo = (uintptr_t)a.p <= (uintptr_t)b.p ? a : b, &hi = &lo == &a ? b : a;
  const uint64_t d = (uintptr_t)hi.p - (uintptr_t)lo.p;
  if (d >= (uint64_t)((lo.rows - 1) * lo.ld + lo.width)) return false;
  if (lo.rows > 1 && hi.rows > 1 && lo.ld != hi.ld) return true;
  const uint64_t ld = lo.rows > 1 ? lo.ld : hi.rows > 1 ? hi.ld : 1;
  return d % ld < (uint64_t)lo.width || d % ld + hi.width > ld;
}
template <typename... S>
inline bool meets(const Span& out, const S&... others) { return (meet(out, others) || ...); }

}  // namespace span_of
}  // namespace qmv

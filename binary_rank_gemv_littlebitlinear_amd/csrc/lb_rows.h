// Whether two strided arrays share memory (host arithmetic only).
#pragma once
#include <cstddef>
#include <cstdint>

namespace lbi {

// Whether the np bytes at p and the nq bytes at q share any.
inline bool overlaps(const void *p, size_t np, const void *q, size_t nq) {
  const char *a = (const char *)p, *b = (const char *)q;
  return a < b + nq && b < a + np;
}

// `rows` rows of `width` bytes, `pitch` >= width bytes apart (a flat array is
// one row).
struct Rows {
  const void *p;
  int64_t rows;
  size_t pitch, width;
  size_t span() const { return rows > 0 ? (size_t)(rows - 1) * pitch + width : 0; }
};

// Whether two arrays may share a byte: not if one ends before the other
// begins, nor if they are column blocks of one buffer, that is, have the same
// pitch (or a single row) and columns apart.  Rows of different pitches whose
// spans meet count as sharing.
inline bool meet(const Rows &a, const Rows &b) {
  if (a.rows < 1 || b.rows < 1 || !overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const size_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  // where b's rows begin, counted from the beginning of a row of a
  const size_t at = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;
  return !(at >= a.width && at + b.width <= pitch);
}

}  // namespace lbi

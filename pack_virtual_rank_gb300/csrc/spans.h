// spans.h -- internal: the memory an array takes, and whether two arrays overlap.
#pragma once

#include <stdint.h>

namespace relay {

// `rows` rows (none: no memory) of `width` bytes, `pitch` bytes apart.
struct Span {
  uintptr_t lo;
  int64_t rows, width, pitch;
  uintptr_t hi() const { return lo + (uintptr_t)((rows - 1) * pitch + width); }
};
inline Span matrix_span(const void* p, int64_t rows, int64_t width, int64_t pitch) {
  return Span{reinterpret_cast<uintptr_t>(p), p == nullptr || width <= 0 ? 0 : rows, width, pitch};
}
inline Span array_span(const void* p, int64_t bytes) { return matrix_span(p, 1, bytes, bytes); }

// Rows of one pitch lie side by side when their offset in it keeps them apart (column views of one buffer), and
// a single row may lie between another's. Of two pitches only the whole ranges are compared.
inline bool overlap(const Span& a, const Span& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.lo >= b.hi() || b.lo >= a.hi()) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  int64_t off = (int64_t)(b.lo - a.lo) % pitch;
  if (off < 0) off += pitch;
  return off < a.width || off + b.width > pitch;
}

}  // namespace relay

// Overlap checks of the entry points: the bytes that a tensor of a call
// occupies, and whether two of them meet.
#pragma once

#include <cstddef>
#include <cstdint>

namespace polar {

// `rows` windows of `width` bytes, `stride` bytes apart (rows x width of a
// contiguous tensor: one window).
struct Strided {
  const void* p;
  size_t rows, width, stride;
  size_t extent() const { return rows ? (rows - 1) * stride + width : 0; }
};

inline Strided span(const void* p, size_t bytes) { return {p, bytes ? (size_t)1 : 0, bytes, bytes}; }

// True where a byte belongs to both.  Windows of one stride may interleave (q
// and k of one projection's output); of different strides, what lies between
// the first byte and the last counts as occupied.
inline bool meet(const Strided& a, const Strided& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const size_t na = a.extent(), nb = b.extent();
  if (!x || !y || !na || !nb || x >= y + nb || y >= x + na) return false;
  if (a.stride != b.stride || a.rows < 2 || b.rows < 2) return true;
  const size_t s = a.stride;
  const size_t off = y >= x ? (size_t)(y - x) % s : (s - (size_t)(x - y) % s) % s;
  return off < a.width || off + b.width > s;
}

}  // namespace polar

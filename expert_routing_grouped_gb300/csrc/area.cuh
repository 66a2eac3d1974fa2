// area.cuh -- whether two row-strided areas of memory meet, for the argument
// checks of the calls that work on the caller's own tensors.
#pragma once

#include <cstddef>
#include <cstdint>

namespace moe {

// `rows` rows of `bytes` bytes, `stride` bytes apart (bytes <= stride); bytes 0
// or a null p: nothing.
struct Area {
  const void *p;
  size_t rows, bytes, stride;
};

static inline Area area(const void *p, size_t bytes) { return Area{p, 1, bytes, bytes}; }

// Exact where both have one stride, or one of them is a single row (columns of
// one wider tensor do not meet); otherwise areas whose spans meet do.
static inline bool meet(const Area &a, const Area &b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes || !a.rows || !b.rows) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const size_t na = (a.rows - 1) * a.stride + a.bytes, nb = (b.rows - 1) * b.stride + b.bytes;
  if (x >= y + nb || y >= x + na) return false;   // the spans do not meet
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  const size_t s = a.rows > 1 ? a.stride : b.stride;
  if (a.rows == 1 && b.rows == 1) return true;
  // b's first byte within a's row pitch.
  const size_t m = y >= x ? (y - x) % s : (s - (x - y) % s) % s;
  return m < a.bytes || m + b.bytes > s;
}

}  // namespace moe

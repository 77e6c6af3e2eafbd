// fp8_checks.cuh -- argument checks shared by the entry points of the block
// norms, the 8-bit floating-point linears (fp8_api.cu) and the experts
// (moe_api.cu).
#pragma once

#include "fp8_common.cuh"

namespace convrot {
namespace fp8 {

// A row-major array of `rows` rows of `width` bytes, `pitch` bytes apart.
struct Region {
  const void* p;
  int64_t rows, width, pitch;
  size_t span() const { return !p || rows <= 0 || width <= 0 ? 0 : static_cast<size_t>((rows - 1) * pitch + width); }
};
inline Region flat(const void* p, int64_t bytes) { return Region{p, 1, bytes, bytes}; }

// Whether two arrays share a byte. Column slices of one buffer (the same
// pitch, apart within it) do not, although their spans interleave.
inline bool meet(const Region& a, const Region& b) {
  if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.pitch != b.pitch || a.rows == 1 || b.rows == 1) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  const int64_t off = ((d % a.pitch) + a.pitch) % a.pitch;  // b's columns after a's, modulo the pitch
  return off < a.width || a.pitch - off < b.width;
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Most rows of a matrix: the kernels count them in 32 bits and may look as far
// as a tile or a ring of staged rows past the last one.
constexpr int64_t MAX_ROWS = 0x7fff0000;
// Longest K, for the same reason: a warp's steps over K go up to 8192 features
// past the last one.
constexpr int64_t MAX_LENGTH = MAX_ROWS;

// Whether rows * pitch (elements) stays far inside 63 bits.
inline bool sane(int64_t rows, int64_t pitch) { return pitch <= (1ll << 40) && rows <= MAX_ROWS; }

}  // namespace fp8
}  // namespace convrot

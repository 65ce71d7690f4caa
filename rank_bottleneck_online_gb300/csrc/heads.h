// heads.h -- host checks of [T, heads, dim] operands: where they lie and whether they meet.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cstdlib>

namespace boost_gb300 {

// One [T, heads, dim] operand of 2-byte values as it lies in memory (strides in elements).
struct Slice {
  uintptr_t base;
  int64_t T, heads, dim, ts, hs;
  // bytes from the first to behind the last element
  uint64_t extent() const {
    return T * heads == 0 ? 0 : 2ull * ((T - 1) * ts + (heads - 1) * hs + dim);
  }
  bool same(const Slice& o) const {
    return base == o.base && heads == o.heads && (T == 1 || ts == o.ts) &&
           (heads == 1 || hs == o.hs);
  }
  // no two elements coincide: tokens apart by more than a token's heads, or heads by more
  // than a head's tokens
  bool one_to_one() const {
    const int64_t token = (heads - 1) * hs + dim, head = (T - 1) * ts + dim;
    return (heads == 1 || hs >= dim) && (T == 1 || ts >= dim) &&
           (T == 1 || heads == 1 || ts >= token || hs >= head);
  }
};

// Whether |x + i step| >= apart for every i from lo to hi.
inline bool stays_away(int64_t x, int64_t step, int64_t lo, int64_t hi, int64_t apart) {
  if (step == 0) lo = hi = 0;
  const int64_t n = step == 0 ? 0 : -x / step;         // the nearest is one of n - 1 .. n + 1
  for (int64_t i = n - 1; i <= n + 1; ++i)
    if (std::abs(x + std::clamp(i, lo, hi) * step) < apart) return false;
  return true;
}

// Whether two operands, of as many tokens and heads as each has, share no element: disjoint ranges;
// heads side by side in the rows of one packed buffer (the same token stride, and spans that do
// not meet modulo it); or heads that lie between each other's (the same strides, and no pair of
// heads and tokens that meet). The stride of a single token or head says nothing: the other's
// counts.
inline bool disjoint(const Slice& a, const Slice& b) {
  if (a.extent() == 0 || b.extent() == 0) return true;
  if (a.base + a.extent() <= b.base || b.base + b.extent() <= a.base) return true;
  if (a.T > 1 && b.T > 1 && a.ts != b.ts) return false;
  const int64_t ts = a.T > 1 ? a.ts : b.T > 1 ? b.ts : 0;
  const int64_t away = static_cast<int64_t>(b.base) - static_cast<int64_t>(a.base);   // bytes
  if (ts > 0) {
    const int64_t sa = 2 * ((a.heads - 1) * a.hs + a.dim), sb = 2 * ((b.heads - 1) * b.hs + b.dim);
    const int64_t row = 2 * ts;
    // where b's span begins within a's rows
    const int64_t o = (away % row + row) % row;
    if (o >= sa && o + sb <= row) return true;
  }
  if (a.heads > 1 && b.heads > 1 && a.hs != b.hs) return false;
  const int64_t hs = a.heads > 1 ? a.hs : b.hs, dim = std::max(a.dim, b.dim);
  for (int64_t h = 1 - a.heads; h < b.heads; ++h)      // b's head less a's
    if (!stays_away(away / 2 + h * hs, ts, 1 - a.T, b.T - 1, dim)) return false;
  return true;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace boost_gb300

// Argument checks shared by the C-ABI files: address ranges, alignment and
// saturating size products (host code).
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace conv3d {

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi)
  bool empty() const { return hi <= lo; }
};

inline Range range_of(const void* p, long long bytes) {
  Range r;
  if (p && bytes > 0) {
    r.lo = (uintptr_t)p;
    r.hi = r.lo + (uintptr_t)bytes;
  }
  return r;
}

inline bool overlaps(const Range& a, const Range& b) {
  return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Product of non-negative sizes, saturating at 2^62 (every size check
// rejects far smaller values), so no size computation overflows.
constexpr long long kSat = 1LL << 62;
inline long long prod(std::initializer_list<long long> v) {
  long long r = 1;
  for (long long a : v) {
    if (a <= 0) return a < 0 ? kSat : 0;
    r = (r > kSat / a) ? kSat : r * a;
  }
  return r;
}

}  // namespace conv3d

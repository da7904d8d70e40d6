// Pieces of the host-side argument checks shared by the check_* functions.
#pragma once

#include <cstdio>
#include <initializer_list>
#include <string>

#include "validate.h"

namespace bmm {

// Extents are capped so that every byte count below fits in int64 without
// overflow checks at each product.
constexpr int64_t kMaxExtent = int64_t(1) << 40;
constexpr int64_t kMaxBytes = int64_t(1) << 50;

inline Status fail(int code, const char* fmt, long long a = 0, long long b = 0) {
  Status s;
  s.code = code;
  char buf[256];
  std::snprintf(buf, sizeof buf, fmt, a, b);
  s.msg = buf;
  return s;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, int64_t an, const void* b, int64_t bn) {
  if (an <= 0 || bn <= 0) return false;
  uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + uintptr_t(bn) && b0 < a0 + uintptr_t(an);
}

// product of non-negative extents, or -1 when it exceeds kMaxBytes
inline int64_t mul_capped(std::initializer_list<int64_t> xs) {
  __int128 p = 1;
  for (int64_t x : xs) {
    p *= x;
    if (p > kMaxBytes) return -1;
  }
  return int64_t(p);
}

}  // namespace bmm

// Pieces of the checks of matrices that lie in rows.
#pragma once

#include "validate_util.h"

namespace bmm {

inline Status failw(const char* what, int code, const char* fmt, long long a = 0, long long b = 0) {
  Status s = fail(code, fmt, a, b);
  s.msg = std::string(what) + ": " + s.msg;
  return s;
}

// A row-major matrix: `rows` rows of `cols` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, cols, ld;
  const char* name;
  int64_t span() const { return rows > 0 && cols > 0 ? (rows - 1) * ld + cols : 0; }
};

// Whether two matrices share a byte. Rows of one buffer that lie side by side
// (equal ld, columns apart) do not.
inline bool overlaps(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.ld != b.ld || a.ld <= 0) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  // columns from a's to b's first one, in [0, ld)
  const int64_t d = y >= x ? int64_t((y - x) % uintptr_t(a.ld))
                           : (a.ld - int64_t((x - y) % uintptr_t(a.ld))) % a.ld;
  return !(d >= a.cols && a.ld - d >= b.cols);
}

// Every output against every input and every other output.
inline Status disjoint(const char* what, std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto q = o + 1; q != outs.end(); ++q)
      if (overlaps(*o, *q)) {
        Status s = failw(what, BMM_EOVERLAP, "");
        s.msg += std::string(o->name) + " overlaps " + q->name;
        return s;
      }
    for (const Rows& i : ins)
      if (overlaps(*o, i)) {
        Status s = failw(what, BMM_EOVERLAP, "");
        s.msg += std::string(o->name) + " overlaps " + i.name;
        return s;
      }
  }
  return Status{};
}

inline Status all_aligned(const char* what, std::initializer_list<Rows> ps) {
  for (const Rows& r : ps)
    if (!aligned16(r.p)) {
      Status s = failw(what, BMM_EALIGN, "");
      s.msg += std::string(r.name) + " must be 16-byte aligned";
      return s;
    }
  return Status{};
}

inline Status all_given(const char* what, std::initializer_list<Rows> ps) {
  for (const Rows& r : ps)
    if (!r.p && r.span() > 0) {
      Status s = failw(what, BMM_EINVAL, "");
      s.msg += std::string(r.name) + " is null";
      return s;
    }
  return Status{};
}

constexpr int64_t kMaxK = int64_t(1) << 22;    // below it (4-bit operands)
constexpr int64_t kMaxLd = int64_t(1) << 21;   // 32-bit offsets inside a tile's rows; the gated
                                               // block's K is such a distance too (dX, dWg, dWu)
constexpr int64_t kMaxF = int64_t(1) << 20;

inline int elem_size(int32_t t) {
  return t == BMM_ELEM_F32 ? 4 : t == BMM_ELEM_F16 || t == BMM_ELEM_BF16 ? 2 : 0;
}

}  // namespace bmm

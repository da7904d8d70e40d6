// What the extern "C" entry points of the feed-forward operators share.
#pragma once

#include <exception>
#include <string>

#include "ffn.h"
#include "validate.h"

namespace bmm {

inline int report(const Status& st) {
  set_last_error(st.msg);
  return st.code;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return report(Status{});
  set_last_error(std::string(what) + ": " + hipGetErrorString(e) +
                 (e == hipErrorInvalidConfiguration ? " (more tiles than one launch may have)" : ""));
  return BMM_EHIP;
}

// No exception (out of host memory in a message, say) leaves a C entry point.
template <class Fn>
auto guarded(Fn fn) noexcept -> decltype(fn()) {
  try {
    return fn();
  } catch (...) {
    return BMM_EHIP;
  }
}

// Start of the second block of output rows where there is none.
constexpr int64_t kNoRow = int64_t(1) << 62;

inline int64_t padded_width(int64_t F) { return (F + 31) / 32 * 32; }

}  // namespace bmm

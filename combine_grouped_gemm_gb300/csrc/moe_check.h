// Argument checks shared by the files that implement the C ABI.
#pragma once

#include <initializer_list>

#include "moe_internal.h"

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// A call's array in bytes; n is 0 for one that is not there.
struct Span {
  const void* p;
  size_t n;
};

// Whether an output meets any of these arrays. The calls' blocks run in any order, so a result
// written over an input would change what other blocks read.
inline bool meets(const Span& out, std::initializer_list<Span> others) {
  const auto o = reinterpret_cast<uintptr_t>(out.p);
  for (const Span& s : others) {
    const auto b = reinterpret_cast<uintptr_t>(s.p);
    if (out.p && s.p && out.n && s.n && o < b + s.n && b < o + out.n) return true;
  }
  return false;
}

}  // namespace moe

#define MOE_CHECK_CFG(cfg)                   \
  do {                                       \
    if (!(cfg)) return MOE_ERR_INVALID_ARG;  \
    const int rc_ = moe::validate(*(cfg));   \
    if (rc_ != MOE_OK) return rc_;           \
  } while (0)

#define MOE_NEED(p)                                    \
  do {                                                 \
    if (!(p)) return MOE_ERR_INVALID_ARG;              \
    if (!moe::aligned16(p)) return MOE_ERR_MISALIGNED; \
  } while (0)

#define MOE_OPT(p)                                            \
  do {                                                        \
    if ((p) && !moe::aligned16(p)) return MOE_ERR_MISALIGNED; \
  } while (0)

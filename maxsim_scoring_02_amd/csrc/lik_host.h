// Host-side helpers that every C entry point uses (defined in lik_api.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "lik.h"

namespace lik {

// Sets lik_last_error() of this host thread and returns `s`.
lik_status fail(lik_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns LIK_OK.
lik_status ok();

// a*b*c... without overflow (at most 2^56), or -1
int64_t mul_ok(std::initializer_list<int64_t> xs);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Memory that a call reads or writes, for checks of overlap.
struct Span {
  const void* p;
  int64_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// Whether an output shares memory with an input or another output.
template <size_t N, size_t M>
inline bool any_overlap(const Span (&in)[N], const Span (&out)[M]) {
  for (size_t i = 0; i < M; ++i) {
    for (size_t j = 0; j < N; ++j)
      if (overlap(out[i], in[j])) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

// LIK_OK when the current device is a gfx950, else LIK_ERR_UNSUPPORTED.
lik_status check_device();

}  // namespace lik

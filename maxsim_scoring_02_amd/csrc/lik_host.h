// Host-side helpers that every C entry point uses (defined in lik_api.hip).
#pragma once

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

// LIK_OK when the current device is a gfx950, else LIK_ERR_UNSUPPORTED.
lik_status check_device();

}  // namespace lik

// Device-side building blocks of the 8-bit cache: codes and scales.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lik_cache_kernels.h"

namespace lik {

constexpr float kScaleMin = 0x1p-40f, kScaleMax = 0x1p40f, kCodeMax = 448.0f;

__device__ __forceinline__ float cache_wave_max(float v) {
  for (int o = 1; o < 64; o *= 2) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// A stored scale as it counts: within its range, NaN as it is.
__device__ __forceinline__ float clamp_scale(float s) {
  return s < kScaleMin ? kScaleMin : (s > kScaleMax ? kScaleMax : s);
}

// The smallest power of two with amax <= 448 times it: 448 = 1.75 * 2^8, so by
// the bits of amax = f * 2^x, 2^(x - 8) where f <= 1.75 and 2^(x - 7) beyond.
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  const int lo = 127 - 40, hi = 127 + 40;
  e = e < lo ? lo : (e > hi ? hi : e);
  return __uint_as_float((uint32_t)e << 23);
}

// The scale of a block that had `was` and needs `need`: the larger, a power of
// two too where `was` is none; NaN stays.
__device__ __forceinline__ float grown_scale(float was, float need) {
  if (was != was) return was;
  const uint32_t u = __float_as_uint(clamp_scale(was));
  const float up = __uint_as_float((u + 0x7fffffu) & 0xff800000u);
  return up > need ? up : need;
}

__device__ __forceinline__ float from_code(uint32_t c) {
  return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}
// Nearest, ties to even; beyond 448 it stays at 448.
__device__ __forceinline__ uint8_t to_code(float f) {
  f = fminf(fmaxf(f, -kCodeMax), kCodeMax);
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(f, 0.0f, 0, false);
}

}  // namespace lik

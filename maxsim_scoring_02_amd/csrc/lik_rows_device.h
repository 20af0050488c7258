// Device-side building blocks of the row losses: softmax statistics of a row
// of logits and the reductions they need.
//
// A row's exponentials are taken in base 2 relative to the row's maximum m:
//
//   e_c = 2^(z_c c - A),  c = scale log2(e),  A = fl(m c),  Z = sum_c e_c,
//
// one fused multiply-add and one v_exp_f32 per logit.  A is a rounded
// product, so every e_c carries the common factor 2^(mc - A); it cancels in
// q_c = e_c / Z, and the log-sum-exp takes it out again:
//
//   lse = scale m + ln2 (log2 Z - (mc - A)),  mc - A exact by one fma.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lik {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A row's softmax: e_c = exp2(fma(z_c, c, -A)), q_c = e_c / Z.
struct RowSoft {
  float m, c, A, Z;
};

// c and A from a row's maximum.  Where m * c overflows float32 (a row of the
// type's lowest values), logits that differ at all differ by more than any
// exponent, so the power of two that brings m next to 2^64 serves as c: equal
// logits still give 1 and smaller ones 0.  An infinite m gives NaN throughout.
__device__ __forceinline__ RowSoft row_ref(float m, float scale) {
  RowSoft r;
  r.m = m;
  r.c = scale * kLog2e;
  r.A = m * r.c;
  if (!(fabsf(r.A) < 1e38f) && fabsf(m) < __builtin_inff()) {
    r.c = ldexpf(1.0f, 64 - ilogbf(m));
    r.A = m * r.c;
  }
  r.Z = 0.0f;
  return r;
}

__device__ __forceinline__ float row_exp(const RowSoft& r, float z) {
  return exp2_fast(fmaf(z, r.c, -r.A));
}

// ln(Z 2^-(mc - A)), the log-sum-exp relative to the maximum.  The logarithm
// is split at the binary exponent, so its error stays near 2^-25 whatever Z.
__device__ __forceinline__ double row_ln_sum(const RowSoft& r) {
  int e;
  float f = frexpf(r.Z, &e);            // [0.5, 1)
  if (f < 0.70710678f) {
    f *= 2.0f;
    --e;
  }
  const double l2 = (double)e + (double)__builtin_amdgcn_logf(f) - (double)fmaf(r.m, r.c, -r.A);
  return kLn2 * l2;
}

// log softmax of one logit of the row
__device__ __forceinline__ double row_logp(const RowSoft& r, float z, float scale, double ln_sum) {
  return (double)scale * ((double)z - (double)r.m) - ln_sum;
}

// Reductions over a workgroup of NT threads; every thread gets the result.
// `tmp` holds NT / 64 values and is free again after the call.
template <int NT, typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* tmp, F f) {
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) v = f(v, __shfl_xor(v, k));
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    v = tmp[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v = f(v, tmp[i]);
    __syncthreads();
  }
  return v;
}

struct MaxF {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumF {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a + b; }
};

// The softmax of a row in two passes over it.  `listed` (or null) is a bitmap
// of columns left out of Z; the maximum is over all columns.
template <int NT, typename T>
__device__ RowSoft row_softmax(const T* __restrict__ row, int64_t C, float scale,
                               const uint32_t* listed, float* tmp) {
  float m = -__builtin_inff();
  for (int64_t c = threadIdx.x; c < C; c += NT) m = fmaxf(m, (float)row[c]);
  m = block_reduce<NT>(m, tmp, MaxF());
  RowSoft r = row_ref(m, scale);
  float z = 0.0f;
  for (int64_t c = threadIdx.x; c < C; c += NT) {
    const float e = row_exp(r, (float)row[c]);
    if (!listed || !(listed[c >> 5] >> (c & 31) & 1)) z += e;
  }
  r.Z = block_reduce<NT>(z, tmp, SumF());
  return r;
}

// Policy loss of one row and its slope dl/dlogp.  x = logp - old, away =
// ref - logp (used with kl != 0 only).
__device__ __forceinline__ void policy_loss(float x, float adv, float low, float high, bool with_kl,
                                            float away, float kl, float* loss, float* slope) {
  const float rho = expf(x);
  const float u = adv == 0.0f ? 0.0f : rho * adv;
  const float v = adv == 0.0f ? 0.0f : fminf(fmaxf(rho, 1.0f - low), 1.0f + high) * adv;
  const bool flows = adv >= 0.0f ? rho <= 1.0f + high : rho >= 1.0f - low;
  float l = u != u ? u : -fminf(u, v);
  float g = flows || u != u ? -u : 0.0f;
  if (with_kl) {
    const float em1 = expm1f(away);
    // exp(d) - d - 1 cancels near 0: its series there
    const float d = away;
    const float series = d * d * (0.5f + d * (1.0f / 6 + d * (1.0f / 24 + d * (1.0f / 120 +
                         d * (1.0f / 720 + d * (1.0f / 5040 + d * (1.0f / 40320)))))));
    l += kl * (fabsf(d) < 0.5f ? series : em1 - d);
    g -= kl * em1;
  }
  *loss = l;
  *slope = g;
}

}  // namespace lik

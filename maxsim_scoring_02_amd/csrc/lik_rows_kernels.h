// Internal interface between the C ABI of the row losses and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lik.h"
#include "lik_rows.h"

namespace lik {

constexpr int64_t kDistillMaxK = 1024;
constexpr int64_t kDistillMaxC = int64_t(1) << 20;   // the bitmap of listed columns fits LDS

inline size_t rows_up(size_t n) { return (n + 255) / 256 * 256; }

// Workspace layout of lik_preference_rows.
struct PrefLayout {
  size_t soft = 0;     // [R] float4 (m, c, A, Z) of each row
  size_t logp = 0;     // [R] double
  size_t coef = 0;     // [R] float, dl/dlogp of each row
  size_t seq = 0;      // [S] double, sequence log-probabilities
  size_t bytes = 0;
};
inline PrefLayout pref_layout(int64_t R, int64_t S) {
  PrefLayout p;
  p.soft = 0;
  p.logp = rows_up(p.soft + (size_t)R * 16);
  p.coef = rows_up(p.logp + (size_t)R * 8);
  p.seq = rows_up(p.coef + (size_t)R * 4);
  p.bytes = rows_up(p.seq + (size_t)S * 8);
  return p;
}

// What every operator takes of its rows.
struct Rows {
  const void* z;
  lik_dtype dtype;
  int64_t R, C, ld;
  float scale;
  void* grad;          // or null
  int64_t grad_ld;
};

hipError_t run_logprob_fwd(const Rows& a, const int32_t* targets, float* logp, float* lse,
                           hipStream_t s);
hipError_t run_logprob_bwd(const Rows& a, const int32_t* targets, const float* lse,
                           const float* grad_logp, hipStream_t s);
hipError_t run_distill(const Rows& a, const int32_t* idx, const float* val, int64_t K,
                       const float* t_lse, const float* weight, float* row_loss, float* loss,
                       hipStream_t s);
hipError_t run_policy(const Rows& a, const int32_t* targets, const float* old_logp,
                      const float* adv, const float* ref, float low, float high, float kl,
                      const float* weight, float* row_loss, float* logp, float* loss,
                      hipStream_t s);

struct PrefArgs {
  const int32_t* targets;
  const int32_t* offsets;
  int64_t S;
  const int32_t* chosen;
  const int32_t* rejected;
  int64_t P;
  const float* ref;
  int kind;
  float beta, margin, smoothing;
  int mean;
  const float* weight;
  float* pair_loss;
  float* seq_logp;
  float* loss;
};
hipError_t run_preference(const Rows& a, const PrefArgs& p, char* ws, hipStream_t s);

}  // namespace lik

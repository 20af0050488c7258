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

// A row cut into parts: part p holds columns [p * cols, (p + 1) * cols), the
// last what is left.  A part is what 256 threads hold in kPartPieces 16-byte
// pieces each at most.
constexpr int kPartPieces = 8;
constexpr int64_t kPartGroups = 512;     // workgroups that fill the chip
struct Parts {
  int cols, n;
};
// At most kPartPieces pieces a thread; fewer while the rows are too few to
// fill the chip.
inline Parts plan_parts(int64_t R, int64_t C, int64_t elem_bytes) {
  const int64_t step = 256 * 16 / elem_bytes;          // one piece a thread
  const int64_t most = (C + step - 1) / step;
  int64_t n = (C + step * kPartPieces - 1) / (step * kPartPieces);
  const int64_t want = (kPartGroups + R - 1) / R;
  if (n < want) n = want < most ? want : most;
  Parts p;
  p.cols = (int)(((C + n - 1) / n + step - 1) / step * step);
  p.n = (int)((C + p.cols - 1) / p.cols);
  return p;
}

inline int64_t elem_bytes_of(lik_dtype t) {
  return t == LIK_F32 ? 4 : (t == LIK_F16 || t == LIK_BF16 ? 2 : 0);
}

// Workspace layouts.
struct RowsLayout {
  size_t parts = 0;    // [R][n] float2 (m, Z)
  size_t soft = 0;     // preference: [R] float4 (m, c, A, Z) of each row
  size_t logp = 0;     // preference: [R] double
  size_t coef = 0;     // preference: [R] float, dl/dlogp of each row
  size_t seq = 0;      // preference: [S] double, sequence log-probabilities
  size_t bytes = 0;
};
inline RowsLayout parts_layout(int64_t R, int64_t C, lik_dtype dtype) {
  RowsLayout w;
  w.bytes = rows_up((size_t)R * plan_parts(R, C, elem_bytes_of(dtype)).n * 8);
  return w;
}
inline RowsLayout pref_layout(int64_t R, int64_t C, int64_t S, lik_dtype dtype) {
  RowsLayout w = parts_layout(R, C, dtype);
  w.soft = w.bytes;
  w.logp = rows_up(w.soft + (size_t)R * 16);
  w.coef = rows_up(w.logp + (size_t)R * 8);
  w.seq = rows_up(w.coef + (size_t)R * 4);
  w.bytes = rows_up(w.seq + (size_t)S * 8);
  return w;
}

// Whether a fused operator holds whole rows in registers, each read once, or
// takes them in parts with a second look for the gradient.
bool rows_held(int64_t R, int64_t C, lik_dtype dtype);

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
                           char* ws, hipStream_t s);
hipError_t run_logprob_bwd(const Rows& a, const int32_t* targets, const float* lse,
                           const float* grad_logp, hipStream_t s);
hipError_t run_distill(const Rows& a, const int32_t* idx, const float* val, int64_t K,
                       const float* t_lse, const float* weight, float* row_loss, float* loss,
                       char* ws, hipStream_t s);
hipError_t run_policy(const Rows& a, const int32_t* targets, const float* old_logp,
                      const float* adv, const float* ref, float low, float high, float kl,
                      const float* weight, float* row_loss, float* logp, float* loss,
                      char* ws, hipStream_t s);

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
// Parts (m, Z) of every row that is not left out: by a negative target, a
// weight of 0, or lying outside the sequences (each where given).
hipError_t run_parts(const Rows& a, const Parts& p, const int32_t* targets, const float* weight,
                     const int32_t* offsets, int64_t S, float2* out, hipStream_t s);

hipError_t run_preference(const Rows& a, const PrefArgs& p, char* ws, hipStream_t s);

}  // namespace lik

// Internal interface between the C ABI of the row losses and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lik.h"
#include "lik_rows.h"

namespace lik {

constexpr int64_t kDistillMaxK = 1024;
// The widest rows that are tested; a listed column's word would hold 2^24 of them.
constexpr int64_t kDistillMaxC = int64_t(1) << 20;
// Sequences times pairs of a preference loss: every sequence looks through the
// pairs for its own, 8.4 ms at 2^34, which atomics would save, and the order of
// the sums with them.
constexpr int64_t kPrefMaxProduct = int64_t(1) << 40;

inline size_t rows_up(size_t n) { return (n + 255) / 256 * 256; }

// A row cut into parts: part p holds columns [p * cols, (p + 1) * cols), the
// last what is left.  A part is taken by a group of gt threads (one wave or 256
// threads) with at most `pieces` 16-byte pieces each.
struct Parts {
  int cols, n, gt;
};
constexpr int64_t kPartGroups = 512;     // workgroups that fill the chip (256 and 1024: no faster)
// Rows that one wave's registers hold go to one wave whole, four rows a workgroup
// (bf16 log-probabilities, 256 threads a row in brackets: 65536 x 300 24 us (81),
// 16384 x 2000 11.8 (21.6), 8192 x 4000 10.9 (14.2)).  Longer ones are cut into as
// few parts as hold them, or more while the rows are too few to fill the chip.
inline Parts plan_parts(int64_t R, int64_t C, int64_t elem_bytes, int pieces) {
  Parts p;
  const int64_t wave = 64 * 16 / elem_bytes;
  if (C <= wave * pieces) {
    p.cols = (int)C;
    p.n = 1;
    p.gt = 64;
    return p;
  }
  const int64_t step = 256 * 16 / elem_bytes;          // one piece a thread
  const int64_t most = (C + step - 1) / step;
  int64_t n = (C + step * pieces - 1) / (step * pieces);
  const int64_t want = (kPartGroups + R - 1) / R;
  if (n < want) n = want < most ? want : most;
  p.cols = (int)(((C + n - 1) / n + step - 1) / step * step);
  p.n = (int)((C + p.cols - 1) / p.cols);
  p.gt = 256;
  return p;
}

// Pieces a thread holds at the first look (4096 x 100003 bf16
// log-probabilities: 2, 4, 8, 16 pieces 164, 130, 124, 133 us) and at most at
// the second (gradients).
constexpr int kLookPieces = 8;
constexpr int kGradPieces = 4;

// Logits that with their gradient exceed the 256 MB cache behind the L2s are
// read and written past the caches; less stays there for what comes next.  With
// other tensors in between, as in training: gradient of 2048 x 50001 f16
// log-probabilities (205 MB) 68 us past the caches, 72 through them; of
// 4096 x 100003 bf16 (819 MB) 284 against 298; preference of 2000 x 32768 f16
// (131 MB) no difference.
constexpr int64_t kFarBytes = int64_t(128) << 20;

// Whether rows of at most `most` bytes are held on chip, each read once, or
// taken in parts with a second look for the gradient: too few rows leave most
// of the chip idle unless they are short (distillation with the rest's term, in
// parts in brackets: 8 x 32000 bf16 13.5 us (16), 8 x 131072 bf16 21 (16), 64 x
// 100003 bf16 21 (21), 192 x 131072 f32 44 (62); policy 128 x 131072 f32 34 (37)).
// Rows of up to 256 KB fit 1024 threads' registers, up to 512 KB registers and
// LDS, next to a teacher's list of at most kDistillLdsK entries.
constexpr int64_t kRegisterBytes = 16 * 1024 * 16;
constexpr int64_t kHeldBytes = 32 * 1024 * 16;
constexpr int64_t kDistillLdsK = 700;

// LDS of a teacher's list of K entries for a group of `threads` (TeacherList), and
// of a held distillation kernel: `held` 16-byte pieces a thread and the lists of a
// workgroup's groups (four of one wave).
constexpr size_t teacher_bytes(int64_t K, int threads) {
  return ((size_t)K * 16 + 4 + (size_t)threads * 4 + 15) / 16 * 16;
}
constexpr size_t distill_lds(int64_t K, int threads, int held) {
  return (size_t)held * threads * 16 + teacher_bytes(K, threads) * (threads == 64 ? 4 : 1);
}
// Beyond kDefaultLds a kernel has to be allowed its LDS, an attribute that it has
// once for all host threads.  So each call sets the most that any call of that
// kernel takes: less would bind another thread's call between its setting and its
// launch.
constexpr size_t kDefaultLds = 65536;
constexpr size_t distill_lds_most(int threads, int held) {
  return distill_lds(held ? kDistillLdsK : kDistillMaxK, threads, held);
}

inline int64_t elem_bytes_of(lik_dtype t) {
  return t == LIK_F32 ? 4 : (t == LIK_F16 || t == LIK_BF16 ? 2 : 0);
}

inline Parts look_parts(int64_t R, int64_t C, lik_dtype dtype) {
  return plan_parts(R, C, elem_bytes_of(dtype), kLookPieces);
}
// Large gradients run best with two pieces a thread (4096 x 100003 bf16 270 us
// against 284 with four), those that stay in the cache with four (2048 x 50001
// f16 63 us against 67).
inline Parts grad_parts(int64_t R, int64_t C, lik_dtype dtype) {
  const int64_t b = elem_bytes_of(dtype);
  return plan_parts(R, C, b, R * C * b > kFarBytes ? 2 : kGradPieces);
}

inline bool rows_held(int64_t R, int64_t C, lik_dtype dtype, int64_t most) {
  const int64_t bytes = C * elem_bytes_of(dtype);
  return bytes <= most && (R >= 128 || bytes <= 65536);
}

// Log-probabilities in one launch: rows of one part, and rows of up to 256 KB by
// 1024 threads while every row has a CU of its own.  bf16, in two launches in
// brackets: 1 x 32000 9.1 us (12.3), 8 x 131072 9.2 (12.1), 256 x 65536 9.2 (13),
// 256 x 131072 14.6 (14.5); 1024 x 131072 52 (44), 4096 x 32000 47 (43).
inline bool logprob_held(int64_t R, int64_t C, lik_dtype dtype) {
  return look_parts(R, C, dtype).n == 1 ||
         (R <= 256 && C * elem_bytes_of(dtype) <= kRegisterBytes);
}

// Workspace layouts.
struct RowsLayout {
  size_t parts = 0;    // [R][n] float2 (m, Z)
  size_t soft = 0;     // preference: [R] float4 (m, c, A, Z) of each row
  size_t coef = 0;     // preference: [R] float, dl/dlogp of each row
  size_t seq = 0;      // preference: [S] double, sequence log-probabilities
  size_t bytes = 0;
};
inline RowsLayout parts_layout(int64_t R, int64_t C, lik_dtype dtype) {
  RowsLayout w;
  w.bytes = rows_up((size_t)R * look_parts(R, C, dtype).n * 8);
  return w;
}
inline RowsLayout pref_layout(int64_t R, int64_t C, int64_t S, lik_dtype dtype) {
  RowsLayout w = parts_layout(R, C, dtype);
  w.soft = w.bytes;
  w.coef = rows_up(w.soft + (size_t)R * 16);
  w.seq = rows_up(w.coef + (size_t)R * 4);
  w.bytes = rows_up(w.seq + (size_t)S * 8);
  return w;
}

// What every operator takes of its rows.
struct Rows {
  const void* z;
  lik_dtype dtype;
  int64_t R, C, ld;
  float scale;
  void* grad;          // or null
  int64_t grad_ld;
  bool far() const { return R * C * elem_bytes_of(dtype) > kFarBytes; }
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

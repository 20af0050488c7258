// C ABI of the row losses (include/lik_rows.h): argument checks and dispatch.
#include <hip/hip_runtime.h>

#include "lik.h"
#include "lik_host.h"
#include "lik_rows.h"
#include "lik_rows_kernels.h"

namespace {

using lik::aligned16;
using lik::aligned4;
using lik::check_device;
using lik::fail;
using lik::mul_ok;
using lik::ok;

constexpr int64_t kMaxRows = INT32_MAX;

// What every operator checks: sizes, type, scale, logits and gradient.
// `done` is set when there is nothing to do.
lik_status check_rows(const lik::Rows& a, bool need_grad, bool* done) {
  *done = false;
  const int64_t size = lik::elem_bytes_of(a.dtype);
  if (!size) return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d for logits", (int)a.dtype);
  if (a.R < 0 || a.C < 0)
    return fail(LIK_ERR_INVALID_ARG, "negative size (R %lld, C %lld)", (long long)a.R,
                (long long)a.C);
  if (a.R == 0) {
    *done = true;
    return LIK_OK;
  }
  if (a.C == 0) return fail(LIK_ERR_INVALID_ARG, "rows have no columns (C == 0)");
  if (a.ld < a.C)
    return fail(LIK_ERR_INVALID_ARG, "row stride ld %lld is less than C %lld", (long long)a.ld,
                (long long)a.C);
  if (a.grad && a.grad_ld < a.C)
    return fail(LIK_ERR_INVALID_ARG, "row stride grad_ld %lld is less than C %lld",
                (long long)a.grad_ld, (long long)a.C);
  if (mul_ok({a.R, a.ld, size}) < 0 || (a.grad && mul_ok({a.R, a.grad_ld, size}) < 0))
    return fail(LIK_ERR_INVALID_ARG, "R x row stride overflows");
  if (a.R > kMaxRows || a.C > kMaxRows)
    return fail(LIK_ERR_UNSUPPORTED, "R and C must be below 2^31 (got %lld, %lld)",
                (long long)a.R, (long long)a.C);
  if (!a.z) return fail(LIK_ERR_INVALID_ARG, "logits is NULL");
  if (need_grad && !a.grad) return fail(LIK_ERR_INVALID_ARG, "grad is NULL");
  const uintptr_t z0 = reinterpret_cast<uintptr_t>(a.z), g0 = reinterpret_cast<uintptr_t>(a.grad);
  if (z0 % size || g0 % size)
    return fail(LIK_ERR_INVALID_ARG, "logits and grad must be aligned to their elements");
  if (!(a.scale >= 0x1p-64f && a.scale <= 0x1p64f))
    return fail(LIK_ERR_INVALID_ARG, "scale must be within [2^-64, 2^64]");
  if (a.grad) {
    const uintptr_t z1 = z0 + (size_t)((a.R - 1) * a.ld + a.C) * size;
    const uintptr_t g1 = g0 + (size_t)((a.R - 1) * a.grad_ld + a.C) * size;
    if (z0 < g1 && g0 < z1) return fail(LIK_ERR_INVALID_ARG, "grad overlaps the logits");
  }
  return LIK_OK;
}

// A required pointer of 4-byte elements.
lik_status need4(const void* p, const char* name) {
  if (!p) return fail(LIK_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned4(p)) return fail(LIK_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return LIK_OK;
}
// One that may be NULL.
lik_status maybe4(const void* p, const char* name) {
  if (!aligned4(p)) return fail(LIK_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return LIK_OK;
}

lik_status check_workspace(size_t need, const void* ws, size_t ws_bytes) {
  if (need == SIZE_MAX) return fail(LIK_ERR_INVALID_ARG, "sizes overflow");
  if (need == 0) return LIK_OK;
  if (!ws || ws_bytes < need)
    return fail(LIK_ERR_INVALID_ARG, "workspace too small: %zu bytes needed, %zu given", need,
                ws ? ws_bytes : (size_t)0);
  if (!aligned16(ws)) return fail(LIK_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return LIK_OK;
}
lik_status check_workspace(lik_rows_op op, const lik::Rows& a, int64_t S, const void* ws,
                           size_t ws_bytes) {
  return check_workspace(lik_rows_workspace_bytes(op, a.R, a.C, S, a.dtype, a.grad ? 1 : 0), ws,
                         ws_bytes);
}

lik_status launched(hipError_t e) {
  if (e != hipSuccess) return fail(LIK_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
  return ok();
}

bool finite(float x) { return x - x == 0.0f; }

}  // namespace

#define LIK_TRY(x)                     \
  do {                                 \
    const lik_status st_ = (x);        \
    if (st_ != LIK_OK) return st_;     \
  } while (0)

extern "C" {

size_t lik_rows_workspace_bytes(lik_rows_op op, int64_t R, int64_t C, int64_t n_seqs,
                                lik_dtype dtype, int flags) {
  const int64_t size = lik::elem_bytes_of(dtype);
  if (!size || R < 0 || C < 0 || mul_ok({R, C, size}) < 0 || mul_ok({R, 64}) < 0) return SIZE_MAX;
  if (R > kMaxRows || C > kMaxRows) return SIZE_MAX;
  switch (op) {
    case LIK_ROWS_LOGPROB_BWD:
      return 0;
    case LIK_ROWS_LOGPROB_FWD:
      if (R == 0 || C == 0 || lik::logprob_held(R, C, dtype)) return 0;
      return lik::parts_layout(R, C, dtype).bytes;
    case LIK_ROWS_DISTILL:
    case LIK_ROWS_POLICY:
      if (R == 0 || C == 0) return 0;
      // a long teacher's list takes the longest rows in parts
      if ((flags & 1) &&
          lik::rows_held(R, C, dtype, op == LIK_ROWS_POLICY ? lik::kHeldBytes : lik::kRegisterBytes))
        return 0;
      return lik::parts_layout(R, C, dtype).bytes;
    case LIK_ROWS_PREFERENCE:
      if (n_seqs < 0 || mul_ok({n_seqs, 64}) < 0) return SIZE_MAX;
      return R == 0 || C == 0 ? 0 : lik::pref_layout(R, C, n_seqs, dtype).bytes;
    case LIK_ROWS_VERIFY:
      if (n_seqs < 0 || n_seqs > kMaxRows) return SIZE_MAX;
      return R == 0 || C == 0 ? 0 : lik::verify_layout(R, C, n_seqs, dtype, flags & 1).bytes;
  }
  return SIZE_MAX;
}

lik_status lik_logprob_rows_fwd(const void* logits, lik_dtype dtype, int64_t R, int64_t C,
                                int64_t ld, const int32_t* targets, float scale, float* logp,
                                float* lse, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const lik::Rows a{logits, dtype, R, C, ld, scale, nullptr, 0};
  bool done;
  LIK_TRY(check_rows(a, false, &done));
  if (done) return ok();
  LIK_TRY(need4(targets, "targets"));
  LIK_TRY(need4(logp, "logp"));
  LIK_TRY(need4(lse, "lse"));
  LIK_TRY(check_workspace(LIK_ROWS_LOGPROB_FWD, a, 0, workspace, workspace_bytes));
  LIK_TRY(check_device());
  return launched(lik::run_logprob_fwd(a, targets, logp, lse, static_cast<char*>(workspace),
                                       static_cast<hipStream_t>(stream)));
}

lik_status lik_logprob_rows_bwd(const void* logits, lik_dtype dtype, int64_t R, int64_t C,
                                int64_t ld, const int32_t* targets, float scale, const float* lse,
                                const float* grad_logp, void* grad, int64_t grad_ld,
                                void* stream) {
  const lik::Rows a{logits, dtype, R, C, ld, scale, grad, grad_ld};
  bool done;
  LIK_TRY(check_rows(a, true, &done));
  if (done) return ok();
  LIK_TRY(need4(targets, "targets"));
  LIK_TRY(need4(lse, "lse"));
  LIK_TRY(need4(grad_logp, "grad_logp"));
  LIK_TRY(check_device());
  return launched(
      lik::run_logprob_bwd(a, targets, lse, grad_logp, static_cast<hipStream_t>(stream)));
}

lik_status lik_distill_rows(const void* logits, lik_dtype dtype, int64_t R, int64_t C, int64_t ld,
                            const int32_t* teacher_idx, const float* teacher_val, int64_t K,
                            const float* teacher_lse, float scale, const float* row_weight,
                            float* row_loss, float* loss, void* grad, int64_t grad_ld,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const lik::Rows a{logits, dtype, R, C, ld, scale, grad, grad_ld};
  bool done;
  LIK_TRY(check_rows(a, false, &done));
  if (K < 0) return fail(LIK_ERR_INVALID_ARG, "negative K %lld", (long long)K);
  if (done) return ok();
  if (mul_ok({R, K, 4}) < 0) return fail(LIK_ERR_INVALID_ARG, "R x K overflows");
  if (K > lik::kDistillMaxK)
    return fail(LIK_ERR_UNSUPPORTED, "distillation supports K <= %lld (got %lld)",
                (long long)lik::kDistillMaxK, (long long)K);
  if (C > lik::kDistillMaxC)
    return fail(LIK_ERR_UNSUPPORTED, "distillation supports C <= %lld (got %lld)",
                (long long)lik::kDistillMaxC, (long long)C);
  if (K > 0) {
    LIK_TRY(need4(teacher_idx, "teacher_idx"));
    LIK_TRY(need4(teacher_val, "teacher_val"));
  }
  LIK_TRY(maybe4(teacher_lse, "teacher_lse"));
  LIK_TRY(maybe4(row_weight, "row_weight"));
  LIK_TRY(need4(row_loss, "row_loss"));
  LIK_TRY(need4(loss, "loss"));
  LIK_TRY(check_workspace(LIK_ROWS_DISTILL, a, 0, workspace, workspace_bytes));
  LIK_TRY(check_device());
  return launched(lik::run_distill(a, teacher_idx, teacher_val, K, teacher_lse, row_weight,
                                   row_loss, loss, static_cast<char*>(workspace),
                                   static_cast<hipStream_t>(stream)));
}

lik_status lik_policy_rows(const void* logits, lik_dtype dtype, int64_t R, int64_t C, int64_t ld,
                           const int32_t* targets, const float* old_logp, const float* advantage,
                           const float* ref_logp, float scale, float clip_low, float clip_high,
                           float kl_coef, const float* row_weight, float* row_loss, float* logp,
                           float* loss, void* grad, int64_t grad_ld, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const lik::Rows a{logits, dtype, R, C, ld, scale, grad, grad_ld};
  bool done;
  LIK_TRY(check_rows(a, false, &done));
  if (!(clip_low >= 0.0f && clip_low <= 1.0f))
    return fail(LIK_ERR_INVALID_ARG, "clip_low must be within [0, 1]");
  if (!(clip_high >= 0.0f)) return fail(LIK_ERR_INVALID_ARG, "clip_high must be at least 0");
  if (!finite(kl_coef)) return fail(LIK_ERR_INVALID_ARG, "kl_coef must be finite");
  if (done) return ok();
  LIK_TRY(need4(targets, "targets"));
  LIK_TRY(need4(old_logp, "old_logp"));
  LIK_TRY(need4(advantage, "advantage"));
  LIK_TRY(maybe4(ref_logp, "ref_logp"));
  LIK_TRY(maybe4(row_weight, "row_weight"));
  LIK_TRY(need4(row_loss, "row_loss"));
  LIK_TRY(need4(logp, "logp"));
  LIK_TRY(need4(loss, "loss"));
  LIK_TRY(check_workspace(LIK_ROWS_POLICY, a, 0, workspace, workspace_bytes));
  LIK_TRY(check_device());
  return launched(lik::run_policy(a, targets, old_logp, advantage, ref_logp, clip_low, clip_high,
                                  kl_coef, row_weight, row_loss, logp, loss,
                                  static_cast<char*>(workspace),
                                  static_cast<hipStream_t>(stream)));
}

lik_status lik_preference_rows(const void* logits, lik_dtype dtype, int64_t R, int64_t C,
                               int64_t ld, const int32_t* targets, const int32_t* seq_offsets,
                               int64_t S, const int32_t* chosen, const int32_t* rejected,
                               int64_t P, const float* ref_logp, lik_pref_kind kind, float beta,
                               float margin, float smoothing, int mean_logp, float scale,
                               const float* pair_weight, float* pair_loss, float* seq_logp,
                               float* loss, void* grad, int64_t grad_ld, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const lik::Rows a{logits, dtype, R, C, ld, scale, grad, grad_ld};
  bool done;
  LIK_TRY(check_rows(a, false, &done));
  if (S < 0 || P < 0) return fail(LIK_ERR_INVALID_ARG, "negative size (S %lld, P %lld)",
                                  (long long)S, (long long)P);
  if (kind != LIK_PREF_SIGMOID && kind != LIK_PREF_HINGE && kind != LIK_PREF_SQUARE)
    return fail(LIK_ERR_INVALID_ARG, "unknown kind %d", (int)kind);
  if (!(beta > 0.0f) || !finite(beta))
    return fail(LIK_ERR_INVALID_ARG, "beta must be finite and positive");
  if (!finite(margin)) return fail(LIK_ERR_INVALID_ARG, "margin must be finite");
  if (!(smoothing >= 0.0f && smoothing <= 0.5f))
    return fail(LIK_ERR_INVALID_ARG, "smoothing must be within [0, 0.5]");
  if (kind != LIK_PREF_SIGMOID && smoothing != 0.0f)
    return fail(LIK_ERR_INVALID_ARG, "smoothing belongs to LIK_PREF_SIGMOID");
  if (kind == LIK_PREF_SQUARE && margin != 0.0f)
    return fail(LIK_ERR_INVALID_ARG, "LIK_PREF_SQUARE has no margin");
  if (done) return ok();
  if (S > kMaxRows || P > kMaxRows)
    return fail(LIK_ERR_UNSUPPORTED, "S and P must be below 2^31");
  if (S > 0 && P > lik::kPrefMaxProduct / S)
    return fail(LIK_ERR_UNSUPPORTED, "S x P must be at most 2^40 (got %lld x %lld)", (long long)S,
                (long long)P);
  LIK_TRY(need4(targets, "targets"));
  LIK_TRY(need4(seq_offsets, "seq_offsets"));
  if (P > 0) {
    LIK_TRY(need4(chosen, "chosen"));
    LIK_TRY(need4(rejected, "rejected"));
    LIK_TRY(need4(pair_loss, "pair_loss"));
  }
  LIK_TRY(maybe4(ref_logp, "ref_logp"));
  LIK_TRY(maybe4(pair_weight, "pair_weight"));
  if (S > 0) LIK_TRY(need4(seq_logp, "seq_logp"));
  LIK_TRY(need4(loss, "loss"));
  LIK_TRY(check_workspace(LIK_ROWS_PREFERENCE, a, S, workspace, workspace_bytes));
  LIK_TRY(check_device());
  const lik::PrefArgs p{targets, seq_offsets, S, chosen, rejected, P, ref_logp, (int)kind, beta,
                        margin, smoothing, mean_logp != 0, pair_weight, pair_loss, seq_logp, loss};
  return launched(lik::run_preference(a, p, static_cast<char*>(workspace),
                                      static_cast<hipStream_t>(stream)));
}

lik_status lik_verify_rows(const void* logits, lik_dtype dtype, int64_t R, int64_t C, int64_t ld,
                           const void* draft_logits, int64_t draft_ld,
                           const int32_t* draft_tokens, const int32_t* seq_offsets, int64_t S,
                           float scale, float draft_scale, const float* accept_u,
                           const float* sample_u, int32_t* tokens, int32_t* accepted, float* logp,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const lik::Rows a{logits, dtype, R, C, ld, scale, nullptr, 0};
  bool done;
  LIK_TRY(check_rows(a, false, &done));
  if (S < 0) return fail(LIK_ERR_INVALID_ARG, "negative size (S %lld)", (long long)S);
  if (!(draft_scale >= 0x1p-64f && draft_scale <= 0x1p64f))
    return fail(LIK_ERR_INVALID_ARG, "draft_scale must be within [2^-64, 2^64]");
  if (done) return ok();
  if (S > kMaxRows) return fail(LIK_ERR_UNSUPPORTED, "S must be below 2^31");
  const int64_t size = lik::elem_bytes_of(dtype);
  if (draft_logits) {
    if (draft_ld < C)
      return fail(LIK_ERR_INVALID_ARG, "row stride draft_ld %lld is less than C %lld",
                  (long long)draft_ld, (long long)C);
    if (mul_ok({R, draft_ld, size}) < 0)
      return fail(LIK_ERR_INVALID_ARG, "R x row stride overflows");
    if (reinterpret_cast<uintptr_t>(draft_logits) % size)
      return fail(LIK_ERR_INVALID_ARG, "draft_logits must be aligned to their elements");
  }
  LIK_TRY(need4(draft_tokens, "draft_tokens"));
  LIK_TRY(need4(seq_offsets, "seq_offsets"));
  LIK_TRY(need4(accept_u, "accept_u"));
  LIK_TRY(need4(tokens, "tokens"));
  LIK_TRY(need4(logp, "logp"));
  if (S > 0) {
    LIK_TRY(need4(sample_u, "sample_u"));
    LIK_TRY(need4(accepted, "accepted"));
  }
  const lik::Span in[] = {{draft_tokens, R * 4}, {accept_u, R * 4}, {seq_offsets, (S + 1) * 4},
                          {sample_u, S * 4},
                          {logits, ((R - 1) * ld + C) * size},
                          {draft_logits, draft_logits ? ((R - 1) * draft_ld + C) * size : 0}};
  const lik::Span out[] = {{tokens, R * 4}, {logp, R * 4}, {accepted, S * 4}};
  if (lik::any_overlap(in, out))
    return fail(LIK_ERR_INVALID_ARG, "an output overlaps an input or another output");
  const size_t need =
      lik_rows_workspace_bytes(LIK_ROWS_VERIFY, R, C, S, dtype, draft_logits ? 1 : 0);
  LIK_TRY(check_workspace(need, workspace, workspace_bytes));
  LIK_TRY(check_device());
  const lik::VerifyArgs v{logits, draft_logits, dtype, R, (int)C, ld, draft_ld, draft_tokens,
                          seq_offsets, S, scale, draft_scale, accept_u, sample_u, tokens,
                          accepted, logp};
  return launched(
      lik::run_verify(v, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"

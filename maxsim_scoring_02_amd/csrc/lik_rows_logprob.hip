// Log-probabilities of rows, their backward, and the preference loss, whose
// gradient needs the log-probabilities of every row of a pair first.
#include <hip/hip_runtime.h>

#include "lik_rows_device.h"
#include "lik_rows_kernels.h"

namespace lik {

namespace {

constexpr int kNT = 256;
constexpr int64_t kMaxGrid = int64_t(1) << 20;

unsigned grid_of(int64_t n) { return (unsigned)(n < kMaxGrid ? n : kMaxGrid); }

template <typename T>
__global__ __launch_bounds__(kNT) void logprob_fwd_kernel(
    const T* __restrict__ z, int64_t R, int64_t C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, float* __restrict__ logp, float* __restrict__ lse) {
  __shared__ float tmp[kNT / 64];
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t t = targets[r];
    float lp = 0.0f, l = 0.0f;
    if (t >= 0) {
      const T* row = z + r * ld;
      const RowSoft s = row_softmax<kNT>(row, C, scale, nullptr, tmp);
      const double ln_sum = row_ln_sum(s);
      lp = t < C ? (float)row_logp(s, (float)row[t], scale, ln_sum) : __builtin_nanf("");
      l = (float)((double)scale * (double)s.m + ln_sum);
    }
    if (threadIdx.x == 0) {
      logp[r] = lp;
      lse[r] = l;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kNT) void logprob_bwd_kernel(
    const T* __restrict__ z, int64_t R, int64_t C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, const float* __restrict__ lse,
    const float* __restrict__ dlogp, T* __restrict__ grad, int64_t gld) {
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t t = targets[r];
    const float d = dlogp[r];
    T* g = grad + r * gld;
    if (t < 0 || d == 0.0f) {
      for (int64_t c = threadIdx.x; c < C; c += kNT) g[c] = (T)0.0f;
      continue;
    }
    const T* row = z + r * ld;
    const float k = t < C ? d * scale : __builtin_nanf("");
    const float l = lse[r];
    for (int64_t c = threadIdx.x; c < C; c += kNT) {
      const float q = exp2_fast(fmaf((float)row[c], scale, -l) * kLog2e);
      g[c] = (T)(c == t ? k - k * q : -k * q);
    }
  }
}

// Rows' softmax statistics and log-probabilities, of rows inside a sequence.
template <typename T>
__global__ __launch_bounds__(kNT) void pref_rows_kernel(
    const T* __restrict__ z, int64_t R, int64_t C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, const int32_t* __restrict__ offsets, int64_t S,
    float4* __restrict__ soft, double* __restrict__ logp, float* __restrict__ coef) {
  __shared__ float tmp[kNT / 64];
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t t = targets[r];
    double lp = 0.0;
    RowSoft s{0, 0, 0, 1};
    if (t >= 0 && r >= offsets[0] && r < offsets[S]) {
      const T* row = z + r * ld;
      s = row_softmax<kNT>(row, C, scale, nullptr, tmp);
      lp = t < C ? row_logp(s, (float)row[t], scale, row_ln_sum(s)) : __builtin_nan("");
    }
    if (threadIdx.x == 0) {
      soft[r] = make_float4(s.m, s.c, s.A, s.Z);
      logp[r] = lp;
      coef[r] = 0.0f;
    }
  }
}

// The rows of a sequence, kept inside [0, R) whatever the offsets say.
__device__ __forceinline__ void seq_range(const int32_t* offsets, int64_t s, int64_t R, int64_t* a,
                                          int64_t* b) {
  const int64_t x = offsets[s], y = offsets[s + 1];
  *a = x < 0 ? 0 : (x > R ? R : x);
  *b = y > R ? R : y;
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) v += __shfl_xor(v, k);
  return v;
}

// One wave per sequence: L_s.
__global__ __launch_bounds__(64) void pref_seq_kernel(PrefArgs p, int64_t R,
                                                      const double* __restrict__ logp,
                                                      double* __restrict__ seq) {
  for (int64_t s = blockIdx.x; s < p.S; s += gridDim.x) {
    int64_t a, b;
    seq_range(p.offsets, s, R, &a, &b);
    double sum = 0.0, n = 0.0;
    for (int64_t r = a + threadIdx.x; r < b; r += 64) {
      sum += logp[r];
      n += p.targets[r] >= 0 ? 1.0 : 0.0;
    }
    sum = wave_sum(sum);
    if (p.mean) {
      n = wave_sum(n);
      if (n > 0.0) sum /= n;
    }
    if (threadIdx.x == 0) {
      seq[s] = sum;
      p.seq_logp[s] = (float)sum;
    }
  }
}

// Loss of one pair and its slope dl/dd; NaN loss and slope 0 for a sequence
// number out of range.
__device__ __forceinline__ void pair_loss(const PrefArgs& p, const double* seq, int64_t i,
                                          double* loss, double* slope) {
  const int32_t c = p.chosen[i], r = p.rejected[i];
  if (c < 0 || r < 0 || c >= p.S || r >= p.S) {
    *loss = __builtin_nan("");
    *slope = 0.0;
    return;
  }
  double d = seq[c] - seq[r];
  if (p.ref) d = (seq[c] - (double)p.ref[c]) - (seq[r] - (double)p.ref[r]);
  const double beta = p.beta;
  const double h = beta * d - (double)p.margin;
  if (p.kind == LIK_PREF_SIGMOID) {
    const double e = p.smoothing;
    const double x = exp(-fabs(h)), tail = log1p(x);
    const double up = h >= 0 ? x / (1 + x) : 1 / (1 + x);     // sigmoid(-h)
    *loss = (1 - e) * (fmax(-h, 0.0) + tail);
    if (e != 0.0) *loss += e * (fmax(h, 0.0) + tail);
    *slope = beta * (e * (1 - up) - (1 - e) * up);
    if (h != h) *loss = h;
  } else if (p.kind == LIK_PREF_HINGE) {
    *loss = h < 1 ? 1 - h : (h != h ? h : 0.0);
    *slope = h < 1 ? -beta : (h != h ? h : 0.0);
  } else {
    const double x = d - 0.5 / beta;
    *loss = x * x;
    *slope = 2 * x;
  }
}

__device__ __forceinline__ double pair_weight(const PrefArgs& p, int64_t i) {
  return p.weight ? (double)p.weight[i] : 1.0 / (double)p.P;
}

// Block 0: the pairs' losses and their sum.  Block 1 + s, one sequence: dl/dL_s
// from every pair it is in, in the pairs' order by lane, onto its rows.
__global__ __launch_bounds__(256) void pref_pairs_kernel(PrefArgs p, int64_t R,
                                                         const double* __restrict__ seq,
                                                         float* __restrict__ coef) {
  __shared__ double tmp[4];
  const int tid = threadIdx.x;
  for (int64_t s = (int64_t)blockIdx.x - 1; s < p.S; s += gridDim.x) {
    if (s < 0) {
      double acc = 0.0;
      for (int64_t i = tid; i < p.P; i += 256) {
        double l, g;
        pair_loss(p, seq, i, &l, &g);
        const double w = pair_weight(p, i);
        p.pair_loss[i] = (float)l;
        if (w != 0.0) acc += w * l;
      }
      acc = block_reduce<256>(acc, tmp, SumF());
      if (tid == 0) *p.loss = (float)acc;
      continue;
    }
    int64_t a, b;
    seq_range(p.offsets, s, R, &a, &b);
    double acc = 0.0;
    for (int64_t i = tid; i < p.P; i += 256) {
      const bool c = p.chosen[i] == s, j = p.rejected[i] == s;
      if (c == j) continue;              // in neither place, or in both
      double l, g;
      pair_loss(p, seq, i, &l, &g);
      const double w = pair_weight(p, i);
      if (w != 0.0) acc += c ? w * g : -w * g;
    }
    acc = block_reduce<256>(acc, tmp, SumF());
    if (p.mean) {
      double n = 0.0;
      for (int64_t r = a + tid; r < b; r += 256) n += p.targets[r] >= 0 ? 1.0 : 0.0;
      n = block_reduce<256>(n, tmp, SumF());
      if (n > 0.0) acc /= n;
    }
    for (int64_t r = a + tid; r < b; r += 256) coef[r] = p.targets[r] >= 0 ? (float)acc : 0.0f;
  }
}

template <typename T>
__global__ __launch_bounds__(kNT) void pref_grad_kernel(
    const T* __restrict__ z, int64_t R, int64_t C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, const float4* __restrict__ soft,
    const float* __restrict__ coef, T* __restrict__ grad, int64_t gld) {
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const float k = coef[r] * scale;
    T* g = grad + r * gld;
    if (k == 0.0f) {
      for (int64_t c = threadIdx.x; c < C; c += kNT) g[c] = (T)0.0f;
      continue;
    }
    const T* row = z + r * ld;
    const int64_t t = targets[r];
    const float4 f = soft[r];
    const RowSoft s{f.x, f.y, f.z, f.w};
    const float kz = -k / s.Z;
    for (int64_t c = threadIdx.x; c < C; c += kNT) {
      const float e = row_exp(s, (float)row[c]);
      g[c] = (T)(c == t ? fmaf(kz, e, k) : kz * e);
    }
  }
}

template <typename T>
hipError_t preference_t(const Rows& a, const PrefArgs& p, char* ws, hipStream_t s) {
  const PrefLayout w = pref_layout(a.R, p.S);
  float4* soft = (float4*)(ws + w.soft);
  double* logp = (double*)(ws + w.logp);
  float* coef = (float*)(ws + w.coef);
  double* seq = (double*)(ws + w.seq);
  hipError_t e;
  if (a.R > 0) {
    hipLaunchKernelGGL(pref_rows_kernel<T>, dim3(grid_of(a.R)), dim3(kNT), 0, s, (const T*)a.z,
                       a.R, a.C, a.ld, a.scale, p.targets, p.offsets, p.S, soft, logp, coef);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (p.S > 0) {
    hipLaunchKernelGGL(pref_seq_kernel, dim3(grid_of(p.S)), dim3(64), 0, s, p, a.R, logp, seq);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(pref_pairs_kernel, dim3(grid_of(p.S + 1)), dim3(256), 0, s, p, a.R, seq,
                     coef);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.grad && a.R > 0) {
    hipLaunchKernelGGL(pref_grad_kernel<T>, dim3(grid_of(a.R)), dim3(kNT), 0, s, (const T*)a.z,
                       a.R, a.C, a.ld, a.scale, p.targets, soft, coef, (T*)a.grad, a.grad_ld);
    e = hipGetLastError();
  }
  return e;
}

template <typename T>
hipError_t logprob_fwd_t(const Rows& a, const int32_t* targets, float* logp, float* lse,
                         hipStream_t s) {
  hipLaunchKernelGGL(logprob_fwd_kernel<T>, dim3(grid_of(a.R)), dim3(kNT), 0, s, (const T*)a.z,
                     a.R, a.C, a.ld, a.scale, targets, logp, lse);
  return hipGetLastError();
}

template <typename T>
hipError_t logprob_bwd_t(const Rows& a, const int32_t* targets, const float* lse,
                         const float* dlogp, hipStream_t s) {
  hipLaunchKernelGGL(logprob_bwd_kernel<T>, dim3(grid_of(a.R)), dim3(kNT), 0, s, (const T*)a.z,
                     a.R, a.C, a.ld, a.scale, targets, lse, dlogp, (T*)a.grad, a.grad_ld);
  return hipGetLastError();
}

}  // namespace

hipError_t run_logprob_fwd(const Rows& a, const int32_t* targets, float* logp, float* lse,
                           hipStream_t s) {
  if (a.dtype == LIK_F16) return logprob_fwd_t<_Float16>(a, targets, logp, lse, s);
  if (a.dtype == LIK_BF16) return logprob_fwd_t<__bf16>(a, targets, logp, lse, s);
  return logprob_fwd_t<float>(a, targets, logp, lse, s);
}

hipError_t run_logprob_bwd(const Rows& a, const int32_t* targets, const float* lse,
                           const float* dlogp, hipStream_t s) {
  if (a.dtype == LIK_F16) return logprob_bwd_t<_Float16>(a, targets, lse, dlogp, s);
  if (a.dtype == LIK_BF16) return logprob_bwd_t<__bf16>(a, targets, lse, dlogp, s);
  return logprob_bwd_t<float>(a, targets, lse, dlogp, s);
}

hipError_t run_preference(const Rows& a, const PrefArgs& p, char* ws, hipStream_t s) {
  if (a.dtype == LIK_F16) return preference_t<_Float16>(a, p, ws, s);
  if (a.dtype == LIK_BF16) return preference_t<__bf16>(a, p, ws, s);
  return preference_t<float>(a, p, ws, s);
}

}  // namespace lik

// Log-probabilities of rows, their backward, and the preference loss, whose
// gradient needs the log-probabilities of every row of a pair first: a first
// look at the rows (parts_kernel), the sequences' and pairs' small sums, and a
// second look that writes the gradient.  The rows are read twice and written
// once; what of them fits the 256 MB cache is read from there the second time.
#include <hip/hip_runtime.h>

#include "lik_rows_device.h"
#include "lik_rows_kernels.h"

namespace lik {

namespace {

// Whether a row has to be read, for the rows' statistics.
__device__ __forceinline__ bool row_counts(int64_t r, const int32_t* targets, const float* weight,
                                           const int32_t* offsets, int64_t S) {
  if (targets && targets[r] < 0) return false;
  if (weight && weight[r] == 0.0f) return false;
  return !offsets || (r >= offsets[0] && r < offsets[S]);
}

// Once: nothing looks at the rows again while they could still be cached.
// Bound by reads: 3584 rows of 100003 bf16 in 104 us, 6.9 TB/s past the caches;
// through them 148 us, 4.8 TB/s.
template <typename T, int GT, bool Once>
__global__ __launch_bounds__(256) void parts_kernel(const T* __restrict__ z, int64_t R, int C,
                                                    int64_t ld, float scale, Parts parts,
                                                    const int32_t* __restrict__ targets,
                                                    const float* __restrict__ weight,
                                                    const int32_t* __restrict__ offsets, int64_t S,
                                                    float2* __restrict__ out) {
  __shared__ float tmp[2 * (GT / 64)];
  const PartAt at = part_at<GT>(parts, C, 0);
  if (at.r >= R || !row_counts(at.r, targets, weight, offsets, S)) return;
  HeldRow<T, GT, kLookPieces, Once> h;
  h.load(z + at.r * ld + at.lo, at.cols, group_tid<GT>(), nullptr);
  const RowSoft s = held_softmax<GT, true>(h, scale, tmp);
  if (group_tid<GT>() == 0) out[at.r * parts.n + at.p] = make_float2(s.m, s.Z);
}

// A row's two outputs.
__device__ __forceinline__ void logprob_write(const RowSoft& s, float zt, float scale, int64_t r,
                                              float* logp, float* lse) {
  const double ln_sum = row_ln_sum(s);
  logp[r] = (float)row_logp(s, zt, scale, ln_sum);
  lse[r] = (float)((double)scale * (double)s.m + ln_sum);
}

// Rows held whole: look and finish in one.
template <typename T, int GT, int NV>
__global__ __launch_bounds__(group_threads<GT>()) void logprob_rows_kernel(
    const T* __restrict__ z, int64_t R, int C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, float* __restrict__ logp, float* __restrict__ lse) {
  __shared__ float tmp[2 * (GT / 64)];
  const int64_t r = group_row<GT>();
  if (r >= R) return;
  const int tid = group_tid<GT>(), t = targets[r];
  if (t < 0) {
    if (tid == 0) logp[r] = lse[r] = 0.0f;
    return;
  }
  const T* row = z + r * ld;
  HeldRow<T, GT, NV> h;
  h.load(row, C, tid, nullptr);
  const float zt = t < C ? (float)row[t] : __builtin_nanf("");
  const RowSoft s = held_softmax<GT>(h, scale, tmp);
  if (tid == 0) logprob_write(s, zt, scale, r, logp, lse);
}

// One wave a row: log-probability and log-sum-exp from the row's parts.
template <typename T>
__global__ __launch_bounds__(256) void logprob_finish_kernel(
    const T* __restrict__ z, int64_t R, int C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, const float2* __restrict__ mz, int n,
    float* __restrict__ logp, float* __restrict__ lse) {
  const int64_t r = group_row<64>();
  if (r >= R) return;
  const int t = targets[r];
  const bool write = (threadIdx.x & 63) == 0;
  if (t < 0) {
    if (write) logp[r] = lse[r] = 0.0f;
    return;
  }
  const float zt = t < C ? (float)z[r * ld + t] : __builtin_nanf("");
  const RowSoft s = merge_parts(mz + r * n, n, scale);
  if (write) logprob_write(s, zt, scale, r, logp, lse);
}

// A part of a row: k ([c == t] - exp(y - lse)).  A stream in and one out: 2048 x
// 50001 f16 in 57 us warm (6.7 TB/s), 66 among other work; 4096 x 100003 bf16 in
// 270 us, 6.0 TB/s.
template <typename T, int GT>
__global__ __launch_bounds__(256) void logprob_bwd_kernel(
    const T* __restrict__ z, int64_t R, int C, int64_t ld, float scale, Parts parts,
    const int32_t* __restrict__ targets, const float* __restrict__ lse,
    const float* __restrict__ dlogp, T* __restrict__ grad, int64_t gld, bool far) {
  const PartAt at = part_at<GT>(parts, C, 0);
  if (at.r >= R) return;
  const int64_t r = at.r;
  const int tid = group_tid<GT>(), t = targets[r];
  const float d = dlogp[r];
  T* g = grad + r * gld + at.lo;
  if (t < 0 || d == 0.0f) {
    fill_row<T, GT>(g, at.cols, tid, 0.0f);
    return;
  }
  const T* row = z + r * ld + at.lo;
  const float k = t < C ? d * scale : __builtin_nanf("");
  const float l = lse[r];
  HeldRow<T, GT, kGradPieces> h;
  h.load(row, at.cols, tid, g);
  // y - lse is rounded once, relative to itself, before it is scaled.  Not above
  // 0, which only the rounding of a very large lse would make it.
  auto prob = [&](float x) {
    const float d = fmaf(x, scale, -l);
    return exp2_fast((d > 0.0f ? 0.0f : d) * kLog2e);
  };
  const int c = t - at.lo;
  const bool mine = c >= 0 && c < at.cols && h.holds(c);
  h.store(g, far, [&](float x) { return -k * prob(x); });
  if (mine) g[c] = (T)fmaf(-k, prob((float)row[c]), k);
}

// The rows of a sequence, kept inside [0, R) whatever the offsets say.
__device__ __forceinline__ void seq_range(const int32_t* offsets, int64_t s, int64_t R, int64_t* a,
                                          int64_t* b) {
  const int64_t x = offsets[s], y = offsets[s + 1];
  *a = x < 0 ? 0 : (x > R ? R : x);
  *b = y > R ? R : y;
}

// What the preference kernels share.
template <typename T>
struct PrefRows {
  const T* z;
  int64_t R, ld;
  int C, n;                // n: parts a row
  float scale;
  const float2* mz;
  float4* soft;
  float* coef;
  double* seq;
};

// Log-probability of a row that counts, its softmax kept for the gradient.
template <typename T>
__device__ __forceinline__ double pref_row(const PrefRows<T>& a, int64_t r, int t) {
  const float zt = t < a.C ? (float)a.z[r * a.ld + t] : __builtin_nanf("");
  const RowSoft f = lane_merge(a.mz + r * a.n, a.n, a.scale);
  a.soft[r] = make_float4(f.m, f.c, f.A, f.Z);
  return row_logp(f, zt, a.scale, row_ln_sum(f));
}

// One workgroup per sequence, a lane per row: L_s.
template <typename T>
__global__ __launch_bounds__(256) void pref_seq_kernel(PrefArgs p, PrefRows<T> a) {
  __shared__ double tmp[4];
  const int64_t s = linear_block();
  if (s >= p.S) return;
  int64_t lo, hi;
  seq_range(p.offsets, s, a.R, &lo, &hi);
  double sum = 0.0, count = 0.0;
  for (int64_t r = lo + threadIdx.x; r < hi; r += 256) {
    const int t = p.targets[r];
    if (t < 0) continue;
    sum += pref_row(a, r, t);
    count += 1.0;
  }
  sum = block_sum(sum, tmp);
  if (p.mean) {
    count = block_sum(count, tmp);
    if (count > 0.0) sum /= count;
  }
  if (threadIdx.x == 0) {
    a.seq[s] = sum;
    p.seq_logp[s] = (float)sum;
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

// What a pair of this slope adds to a sequence that it sets first (c), second (j)
// or against itself: then 0, or NaN where the slope is.
__device__ __forceinline__ double pair_part(double slope, bool c, bool j) {
  return (c ? slope : 0.0) - (j ? slope : 0.0);
}

__device__ __forceinline__ double pair_weight(const PrefArgs& p, int64_t i) {
  return p.weight ? (double)p.weight[i] : 1.0 / (double)p.P;
}

// Block 0: the pairs' losses and their sum.  Block 1 + s, one sequence (for the
// gradient): dl/dL_s from every pair it is in, in the pairs' order by lane, onto
// its rows.
__global__ __launch_bounds__(256) void pref_pairs_kernel(PrefArgs p, int64_t R,
                                                         const double* __restrict__ seq,
                                                         float* __restrict__ coef) {
  __shared__ double tmp[4];
  const int tid = threadIdx.x;
  const int64_t s = linear_block() - 1;
  if (s >= p.S) return;
  if (s < 0) {
    double acc = 0.0;
    for (int64_t i = tid; i < p.P; i += 256) {
      double l, g;
      pair_loss(p, seq, i, &l, &g);
      const double w = pair_weight(p, i);
      p.pair_loss[i] = (float)l;
      if (w != 0.0) acc += w * l;
    }
    acc = block_sum(acc, tmp);
    if (tid == 0) *p.loss = (float)acc;
    return;
  }
  int64_t a, b;
  seq_range(p.offsets, s, R, &a, &b);
  double acc = 0.0, n = 0.0;
  for (int64_t i = tid; i < p.P; i += 256) {
    const bool c = p.chosen[i] == s, j = p.rejected[i] == s;
    if (!c && !j) continue;
    double l, g;
    pair_loss(p, seq, i, &l, &g);
    const double w = pair_weight(p, i);
    if (w != 0.0) acc += pair_part(w * g, c, j);
  }
  acc = block_sum(acc, tmp);
  if (p.mean) {
    for (int64_t r = a + tid; r < b; r += 256) n += p.targets[r] >= 0 ? 1.0 : 0.0;
    n = block_sum(n, tmp);
    if (n > 0.0) acc /= n;
  }
  for (int64_t r = a + tid; r < b; r += 256) coef[r] = p.targets[r] >= 0 ? (float)acc : 0.0f;
}

// Both of the above in one workgroup, for few rows, sequences and pairs: a
// launch less where launches are most of the time (120 rows 5.3 us; at 1999 rows
// 12.7 us where the two above take 4.5 and 4.0).  Sums run in another order than
// in the kernels above, in a fixed one too.
constexpr int kSmallRows = 512, kSmallSeqs = 256, kSmallPairs = 512;
template <typename T>
__global__ __launch_bounds__(1024) void pref_small_kernel(PrefArgs p, PrefRows<T> a) {
  __shared__ double seq[kSmallSeqs], count[kSmallSeqs], slope[kSmallPairs], sums[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  for (int s = wave; s < p.S; s += 16) {
    int64_t lo, hi;
    seq_range(p.offsets, s, a.R, &lo, &hi);
    double sum = 0.0, n = 0.0;
    for (int64_t r = lo + lane; r < hi; r += 64) {
      const int t = p.targets[r];
      if (t < 0) continue;
      sum += pref_row(a, r, t);
      n += 1.0;
    }
    sum = wave_sum(sum);
    n = p.mean ? wave_sum(n) : 1.0;
    if (n == 0.0) n = 1.0;
    sum /= n;
    if (lane == 0) {
      seq[s] = sum;
      count[s] = n;
      p.seq_logp[s] = (float)sum;
    }
  }
  __syncthreads();
  double acc = 0.0;
  if (tid < p.P) {
    double l, g;
    pair_loss(p, seq, tid, &l, &g);
    const double w = pair_weight(p, tid);
    p.pair_loss[tid] = (float)l;
    acc = w != 0.0 ? w * l : 0.0;
    slope[tid] = w != 0.0 ? w * g : 0.0;
  }
  acc = wave_sum(acc);
  if (lane == 0) sums[wave] = acc;
  __syncthreads();
  if (wave == 0) {
    acc = wave_sum(lane < 16 ? sums[lane] : 0.0);
    if (lane == 0) *p.loss = (float)acc;
  }
  for (int s = wave; s < p.S; s += 16) {
    int64_t lo, hi;
    seq_range(p.offsets, s, a.R, &lo, &hi);
    double d = 0.0;
    for (int i = lane; i < p.P; i += 64) {
      const bool c = p.chosen[i] == s, j = p.rejected[i] == s;
      if (c || j) d += pair_part(slope[i], c, j);
    }
    d = wave_sum(d) / count[s];
    for (int64_t r = lo + lane; r < hi; r += 64) a.coef[r] = p.targets[r] >= 0 ? (float)d : 0.0f;
  }
}

// A part of a row's gradient; 0 for rows outside every sequence.  4096 x 100000
// bf16 in 221 us (6.9 TB/s, part of the reads from the cache behind the L2s);
// 2000 x 32768 f16 in 30 us (8.2 TB/s, all of them).
template <typename T, int GT>
__global__ __launch_bounds__(256) void pref_grad_kernel(
    const T* __restrict__ z, int64_t R, int C, int64_t ld, float scale, Parts parts, PrefArgs p,
    const float4* __restrict__ soft, const float* __restrict__ coef, T* __restrict__ grad,
    int64_t gld, bool far) {
  const PartAt at = part_at<GT>(parts, C, 0);
  if (at.r >= R) return;
  const int64_t r = at.r;
  const int tid = group_tid<GT>();
  T* g = grad + r * gld + at.lo;
  const bool in = p.S > 0 && row_counts(r, p.targets, nullptr, p.offsets, p.S);
  const float k = in ? coef[r] * scale : 0.0f;
  if (k == 0.0f) {
    fill_row<T, GT>(g, at.cols, tid, 0.0f);
    return;
  }
  const T* row = z + r * ld + at.lo;
  HeldRow<T, GT, kGradPieces, false> h;      // what the caches kept of the first look
  h.load(row, at.cols, tid, g);
  const float4 f = soft[r];
  const RowSoft s{f.x, f.y, f.z, f.w};
  const float kz = -k / s.Z;
  const int c = p.targets[r] - at.lo;
  const bool mine = c >= 0 && c < at.cols && h.holds(c);
  h.store(g, far, [&](float x) { return kz * row_exp(s, x); });
  if (mine) g[c] = (T)fmaf(kz, row_exp(s, (float)row[c]), k);
}

template <typename T>
hipError_t parts_t(const Rows& a, const Parts& p, bool once, const int32_t* targets,
                   const float* weight, const int32_t* offsets, int64_t S, float2* out,
                   hipStream_t s) {
  return parts_dispatch(p, [&](auto gt) {
    constexpr int GT = decltype(gt)::value;
    const auto kernel = once ? parts_kernel<T, GT, true> : parts_kernel<T, GT, false>;
    hipLaunchKernelGGL(kernel, group_grid<GT>(a.R * p.n), dim3(256), 0, s, (const T*)a.z, a.R,
                       (int)a.C, a.ld, a.scale, p, targets, weight, offsets, S, out);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t preference_t(const Rows& a, const PrefArgs& p, char* ws, hipStream_t s) {
  const RowsLayout w = pref_layout(a.R, a.C, p.S, a.dtype);
  const Parts look = look_parts(a.R, a.C, a.dtype), parts = grad_parts(a.R, a.C, a.dtype);
  float2* mz = (float2*)(ws + w.parts);
  float4* soft = (float4*)(ws + w.soft);
  float* coef = (float*)(ws + w.coef);
  double* seq = (double*)(ws + w.seq);
  const PrefRows<T> rows{(const T*)a.z, a.R, a.ld, (int)a.C, look.n, a.scale, mz, soft, coef, seq};
  hipError_t e;
  if (p.S > 0) {
    e = run_parts(a, look, p.targets, nullptr, p.offsets, p.S, mz, s);
    if (e != hipSuccess) return e;
  }
  if (a.R <= kSmallRows && p.S <= kSmallSeqs && p.P <= kSmallPairs) {
    hipLaunchKernelGGL(pref_small_kernel<T>, dim3(1), dim3(1024), 0, s, p, rows);
  } else {
    if (p.S > 0) {
      hipLaunchKernelGGL(pref_seq_kernel<T>, linear_grid(p.S), dim3(256), 0, s, p, rows);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(pref_pairs_kernel, linear_grid(a.grad ? p.S + 1 : 1), dim3(256), 0, s, p,
                       a.R, seq, coef);
  }
  if ((e = hipGetLastError()) != hipSuccess || !a.grad) return e;
  return parts_dispatch(parts, [&](auto gt) {
    constexpr int GT = decltype(gt)::value;
    hipLaunchKernelGGL((pref_grad_kernel<T, GT>), group_grid<GT>(a.R * parts.n), dim3(256), 0, s,
                       (const T*)a.z, a.R, (int)a.C, a.ld, a.scale, parts, p, soft, coef,
                       (T*)a.grad, a.grad_ld, a.far());
    return hipGetLastError();
  });
}

template <typename T>
hipError_t logprob_fwd_t(const Rows& a, const int32_t* targets, float* logp, float* lse, char* ws,
                         hipStream_t s) {
  const Parts parts = look_parts(a.R, a.C, a.dtype);
  const auto whole = [&](auto gt, auto nv) {
    constexpr int GT = decltype(gt)::value, NV = decltype(nv)::value;
    hipLaunchKernelGGL((logprob_rows_kernel<T, GT, NV>), group_grid<GT>(a.R),
                       dim3(group_threads<GT>()), 0, s, (const T*)a.z, a.R, (int)a.C, a.ld, a.scale,
                       targets, logp, lse);
    return hipGetLastError();
  };
  if (parts.n == 1)
    return parts_dispatch(parts, [&](auto gt) {
      return whole(gt, std::integral_constant<int, kLookPieces>());
    });
  if (logprob_held(a.R, a.C, a.dtype)) {
    const std::integral_constant<int, 1024> gt;
    if (a.C <= HeldRow<T, 1024, 4>::kColumns) return whole(gt, std::integral_constant<int, 4>());
    if (a.C <= HeldRow<T, 1024, 8>::kColumns) return whole(gt, std::integral_constant<int, 8>());
    return whole(gt, std::integral_constant<int, 16>());
  }
  float2* mz = (float2*)ws;
  hipError_t e = parts_t<T>(a, parts, true, targets, nullptr, nullptr, 0, mz, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(logprob_finish_kernel<T>, group_grid<64>(a.R), dim3(256), 0, s,
                     (const T*)a.z, a.R, (int)a.C, a.ld, a.scale, targets, mz, parts.n, logp, lse);
  return hipGetLastError();
}

template <typename T>
hipError_t logprob_bwd_t(const Rows& a, const int32_t* targets, const float* lse,
                         const float* dlogp, hipStream_t s) {
  const Parts parts = grad_parts(a.R, a.C, a.dtype);
  return parts_dispatch(parts, [&](auto gt) {
    constexpr int GT = decltype(gt)::value;
    hipLaunchKernelGGL((logprob_bwd_kernel<T, GT>), group_grid<GT>(a.R * parts.n), dim3(256), 0, s,
                       (const T*)a.z, a.R, (int)a.C, a.ld, a.scale, parts, targets, lse, dlogp,
                       (T*)a.grad, a.grad_ld, a.far());
    return hipGetLastError();
  });
}

}  // namespace

hipError_t run_parts(const Rows& a, const Parts& p, const int32_t* targets, const float* weight,
                     const int32_t* offsets, int64_t S, float2* out, hipStream_t s) {
  // rows that fit the cache behind the L2s stay there for the second look; past
  // it they load faster (4096 x 100000 bf16 105 us against 148)
  const bool once = a.far();
  if (a.dtype == LIK_F16) return parts_t<_Float16>(a, p, once, targets, weight, offsets, S, out, s);
  if (a.dtype == LIK_BF16) return parts_t<__bf16>(a, p, once, targets, weight, offsets, S, out, s);
  return parts_t<float>(a, p, once, targets, weight, offsets, S, out, s);
}

hipError_t run_logprob_fwd(const Rows& a, const int32_t* targets, float* logp, float* lse,
                           char* ws, hipStream_t s) {
  if (a.dtype == LIK_F16) return logprob_fwd_t<_Float16>(a, targets, logp, lse, ws, s);
  if (a.dtype == LIK_BF16) return logprob_fwd_t<__bf16>(a, targets, logp, lse, ws, s);
  return logprob_fwd_t<float>(a, targets, logp, lse, ws, s);
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

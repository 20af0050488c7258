// Row losses whose gradient needs nothing beyond its own row: distillation
// from a teacher's top logits, and the clipped policy loss.
#include <hip/hip_runtime.h>

#include "lik_rows_device.h"
#include "lik_rows_kernels.h"

namespace lik {

namespace {

constexpr int kNT = 256;
constexpr int64_t kMaxGrid = int64_t(1) << 20;

template <int NT, typename T>
__device__ void fill_row(T* __restrict__ g, int64_t C, float v) {
  for (int64_t c = threadIdx.x; c < C; c += NT) g[c] = (T)v;
}

// loss = sum_r w_r l_r, rows of weight 0 left out
__global__ __launch_bounds__(256) void weighted_sum_kernel(const float* __restrict__ l,
                                                           const float* __restrict__ w, int64_t R,
                                                           float* __restrict__ loss) {
  __shared__ double tmp[4];
  double acc = 0.0;
  for (int64_t r = threadIdx.x; r < R; r += 256) {
    const float k = w ? w[r] : 1.0f;
    if (k != 0.0f) acc += (double)k * (double)l[r];
  }
  acc = block_reduce<256>(acc, tmp, SumF());
  if (threadIdx.x == 0) *loss = (float)(w ? acc : acc / (double)R);
}

template <typename T>
__global__ __launch_bounds__(kNT) void policy_rows_kernel(
    const T* __restrict__ z, int64_t R, int64_t C, int64_t ld, float scale,
    const int32_t* __restrict__ targets, const float* __restrict__ old_logp,
    const float* __restrict__ adv, const float* __restrict__ ref, float low, float high, float kl,
    const float* __restrict__ weight, float* __restrict__ row_loss, float* __restrict__ logp,
    T* __restrict__ grad, int64_t gld) {
  __shared__ float tmp[kNT / 64];
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t t = targets[r];
    const float w = weight ? weight[r] : 1.0f / (float)R;
    T* g = grad ? grad + r * gld : nullptr;
    if (t < 0 || w == 0.0f) {
      if (threadIdx.x == 0) row_loss[r] = logp[r] = 0.0f;
      if (g) fill_row<kNT>(g, C, 0.0f);
      continue;
    }
    const T* row = z + r * ld;
    const RowSoft s = row_softmax<kNT>(row, C, scale, nullptr, tmp);
    const float zt = t < C ? (float)row[t] : __builtin_nanf("");
    const double lp = row_logp(s, zt, scale, row_ln_sum(s));
    float l, slope;
    policy_loss((float)(lp - (double)old_logp[r]), adv[r], low, high, ref != nullptr,
                ref ? (float)((double)ref[r] - lp) : 0.0f, kl, &l, &slope);
    if (threadIdx.x == 0) {
      row_loss[r] = l;
      logp[r] = (float)lp;
    }
    if (g) {
      const float k = w * slope * scale;
      const float kz = -k / s.Z;
      for (int64_t c = threadIdx.x; c < C; c += kNT) {
        const float e = row_exp(s, (float)row[c]);
        g[c] = (T)(c == t ? fmaf(kz, e, k) : kz * e);
      }
    }
  }
}

// What the teacher's list says of a row, held in LDS while the row is done.
struct TeacherList {
  int32_t col[kDistillMaxK];    // column, or -1
  int32_t lead[kDistillMaxK];   // 1: first entry of its column
  float p[kDistillMaxK];        // teacher probability
  float zs[kDistillMaxK];       // the student's logit there
};

template <typename T>
__global__ __launch_bounds__(kNT) void distill_rows_kernel(
    const T* __restrict__ z, int64_t R, int64_t C, int64_t ld, float scale,
    const int32_t* __restrict__ idx, const float* __restrict__ val, int K,
    const float* __restrict__ t_lse, const float* __restrict__ weight,
    float* __restrict__ row_loss, T* __restrict__ grad, int64_t gld) {
  __shared__ TeacherList L;
  __shared__ float tmp[kNT / 64];
  __shared__ double tmpd[kNT / 64];
  __shared__ int flags;                     // 1: a column >= C, 2: a column twice, 4: an entry with mass
  extern __shared__ uint32_t listed[];      // bitmap of the listed columns
  const int tid = threadIdx.x;
  const int words = (int)((C + 31) / 32);
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const float w = weight ? weight[r] : 1.0f / (float)R;
    T* g = grad ? grad + r * gld : nullptr;
    if (w == 0.0f) {
      if (tid == 0) row_loss[r] = 0.0f;
      if (g) fill_row<kNT>(g, C, 0.0f);
      continue;
    }
    const T* row = z + r * ld;
    __syncthreads();
    for (int i = tid; i < words; i += kNT) listed[i] = 0;
    if (tid == 0) flags = 0;
    __syncthreads();
    float tmax = -__builtin_inff();
    for (int k = tid; k < K; k += kNT) {
      const int32_t j = idx[r * K + k];
      const float t = val[r * K + k];
      int32_t col = j < 0 ? -1 : j;
      if (j >= C) {
        col = -1;
        atomicOr(&flags, 1);
      }
      L.col[k] = col;
      L.lead[k] = col >= 0;
      L.p[k] = t;
      L.zs[k] = 0.0f;
      if (col >= 0) {
        L.zs[k] = (float)row[col];
        const uint32_t bit = 1u << (col & 31);
        if (atomicOr(&listed[col >> 5], bit) & bit) atomicOr(&flags, 2);
        tmax = fmaxf(tmax, t);
        if (!(t == -__builtin_inff())) atomicOr(&flags, 4);
      }
    }
    __syncthreads();
    if (flags & 2) {
      // a column twice: its first entry stands for it
      for (int k = tid; k < K; k += kNT) {
        int lead = L.col[k] >= 0;
        for (int i = 0; i < k; ++i) lead &= L.col[i] != L.col[k];
        L.lead[k] = lead;
      }
      __syncthreads();
    }
    if (!t_lse && !(flags & 5)) {
      if (tid == 0) row_loss[r] = 0.0f;
      if (g) fill_row<kNT>(g, C, 0.0f);
      continue;
    }
    // teacher probabilities
    double lt;
    if (t_lse) {
      lt = (double)t_lse[r];
    } else {
      tmax = block_reduce<kNT>(tmax, tmp, MaxF());
      float sum = 0.0f;
      for (int k = tid; k < K; k += kNT)
        if (L.col[k] >= 0) sum += expf(scale * (L.p[k] - tmax));
      sum = block_reduce<kNT>(sum, tmp, SumF());
      lt = (double)scale * (double)tmax + (double)logf(sum);
    }
    double mass = 0.0;
    for (int k = tid; k < K; k += kNT) {
      float p = 0.0f;
      if (L.col[k] >= 0 && L.p[k] != -__builtin_inff())
        p = expf((float)((double)scale * (double)L.p[k] - lt));
      if (L.col[k] >= 0) mass += (double)p;
    }
    mass = block_reduce<kNT>(mass, tmpd, SumF());
    // the student's: listed columns apart from the rest
    RowSoft s = row_softmax<kNT>(row, C, scale, listed, tmp);
    const float rest = s.Z;
    double top = 0.0, terms = 0.0, leads = 0.0;
    for (int k = tid; k < K; k += kNT) {
      if (L.col[k] < 0) continue;
      if (L.lead[k]) {
        top += (double)row_exp(s, L.zs[k]);
        leads += 1.0;
      }
      const double lp = (double)scale * (double)L.p[k] - lt;
      const float p = L.p[k] == -__builtin_inff() ? 0.0f : expf((float)lp);
      if (p != 0.0f) terms += (double)p * (lp - (double)scale * ((double)L.zs[k] - (double)s.m));
      L.p[k] = p;
    }
    top = block_reduce<kNT>(top, tmpd, SumF());
    terms = block_reduce<kNT>(terms, tmpd, SumF());
    leads = block_reduce<kNT>(leads, tmpd, SumF());
    s.Z = (float)((double)rest + top);
    const double ln_sum = row_ln_sum(s);
    double l = terms + mass * ln_sum;
    float p_rest = 0.0f;
    if (t_lse && leads < (double)C) {
      p_rest = (float)fmax(0.0, 1.0 - mass);
      if (mass != mass) p_rest = __builtin_nanf("");
      if (p_rest != 0.0f)
        l += (double)p_rest * ((double)logf(p_rest) - (double)logf(rest / s.Z));
    }
    const float nan = flags & 1 ? __builtin_nanf("") : 0.0f;
    if (tid == 0) row_loss[r] = (float)l + nan;
    if (g) {
      const float k = w * scale + nan;
      const float M = (float)(mass + (double)p_rest);
      const float others = rest > 0.0f ? k * (M / s.Z - p_rest / rest) : (rest == 0.0f ? nan : rest);
      const float on = k * (M / s.Z);
      for (int64_t c = tid; c < C; c += kNT)
        if (!(listed[c >> 5] >> (c & 31) & 1)) g[c] = (T)(others * row_exp(s, (float)row[c]));
      __syncthreads();
      for (int i = tid; i < K; i += kNT) {
        if (!L.lead[i]) continue;
        float p = L.p[i];
        if (flags & 2)
          for (int j = i + 1; j < K; ++j)
            if (L.col[j] == L.col[i]) p += L.p[j];
        g[L.col[i]] = (T)(on * row_exp(s, L.zs[i]) - k * p);
      }
    }
  }
}

template <typename T>
hipError_t policy_t(const Rows& a, const int32_t* targets, const float* old_logp, const float* adv,
                    const float* ref, float low, float high, float kl, const float* weight,
                    float* row_loss, float* logp, hipStream_t s) {
  const unsigned grid = (unsigned)(a.R < kMaxGrid ? a.R : kMaxGrid);
  hipLaunchKernelGGL(policy_rows_kernel<T>, dim3(grid), dim3(kNT), 0, s, (const T*)a.z, a.R, a.C,
                     a.ld, a.scale, targets, old_logp, adv, ref, low, high, kl, weight, row_loss,
                     logp, (T*)a.grad, a.grad_ld);
  return hipGetLastError();
}

template <typename T>
hipError_t distill_t(const Rows& a, const int32_t* idx, const float* val, int64_t K,
                     const float* t_lse, const float* weight, float* row_loss, hipStream_t s) {
  const unsigned grid = (unsigned)(a.R < kMaxGrid ? a.R : kMaxGrid);
  const size_t lds = (size_t)((a.C + 31) / 32) * 4;
  hipLaunchKernelGGL(distill_rows_kernel<T>, dim3(grid), dim3(kNT), lds, s, (const T*)a.z, a.R,
                     a.C, a.ld, a.scale, idx, val, (int)K, t_lse, weight, row_loss, (T*)a.grad,
                     a.grad_ld);
  return hipGetLastError();
}

hipError_t weighted_sum(const float* l, const float* w, int64_t R, float* loss, hipStream_t s) {
  hipLaunchKernelGGL(weighted_sum_kernel, dim3(1), dim3(256), 0, s, l, w, R, loss);
  return hipGetLastError();
}

}  // namespace

hipError_t run_policy(const Rows& a, const int32_t* targets, const float* old_logp,
                      const float* adv, const float* ref, float low, float high, float kl,
                      const float* weight, float* row_loss, float* logp, float* loss,
                      hipStream_t s) {
  hipError_t e;
  if (a.dtype == LIK_F16)
    e = policy_t<_Float16>(a, targets, old_logp, adv, ref, low, high, kl, weight, row_loss, logp, s);
  else if (a.dtype == LIK_BF16)
    e = policy_t<__bf16>(a, targets, old_logp, adv, ref, low, high, kl, weight, row_loss, logp, s);
  else
    e = policy_t<float>(a, targets, old_logp, adv, ref, low, high, kl, weight, row_loss, logp, s);
  return e != hipSuccess ? e : weighted_sum(row_loss, weight, a.R, loss, s);
}

hipError_t run_distill(const Rows& a, const int32_t* idx, const float* val, int64_t K,
                       const float* t_lse, const float* weight, float* row_loss, float* loss,
                       hipStream_t s) {
  hipError_t e;
  if (a.dtype == LIK_F16)
    e = distill_t<_Float16>(a, idx, val, K, t_lse, weight, row_loss, s);
  else if (a.dtype == LIK_BF16)
    e = distill_t<__bf16>(a, idx, val, K, t_lse, weight, row_loss, s);
  else
    e = distill_t<float>(a, idx, val, K, t_lse, weight, row_loss, s);
  return e != hipSuccess ? e : weighted_sum(row_loss, weight, a.R, loss, s);
}

}  // namespace lik

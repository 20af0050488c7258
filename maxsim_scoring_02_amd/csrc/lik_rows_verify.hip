// Verification of drafted tokens (include/lik_rows.h, lik_verify_rows).
#include <hip/hip_runtime.h>

#include "lik_rows_device.h"
#include "lik_rows_kernels.h"

namespace lik {

namespace {

// A row's softmax by 256 threads: its maximum, then its sum.
template <typename T>
__device__ RowSoft block_softmax(const T* row, int C, float scale, double* tmp) {
  __shared__ float top[4];
  float m = -kInf;
  for (int c = threadIdx.x; c < C; c += 256) m = fmaxf(m, (float)row[c]);
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) top[wave_id()] = m;
  __syncthreads();
  m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  RowSoft s = row_ref(m, scale);
  double Z = 0.0;
  for (int c = threadIdx.x; c < C; c += 256) Z += (double)row_exp(s, (float)row[c]);
  s.Z = (float)block_sum(Z, tmp);
  if (m == -kInf) s.Z = __builtin_nanf("");
  return s;
}

// One workgroup per sequence, row after row.
template <typename T>
__global__ __launch_bounds__(256) void verify_kernel(VerifyArgs a, const T* z, const T* d) {
  __shared__ double tmp[4], wave_tot[4];
  __shared__ int found;
  const int64_t s = linear_block();
  const int tid = threadIdx.x;
  if (s >= a.S) return;
  int64_t lo = a.offsets[s], hi = a.offsets[s + 1];
  if (lo < 0) lo = 0;
  if (hi > a.R) hi = a.R;
  if (hi <= lo) {
    if (tid == 0) a.accepted[s] = 0;
    return;
  }
  int64_t r = lo;
  for (;; ++r) {
    const int x = a.drafts[r];
    const bool more = r + 1 < hi && x >= 0;
    const T* row = z + r * a.ld;
    const T* drow = d ? d + r * a.draft_ld : nullptr;
    const RowSoft p = block_softmax(row, a.C, a.scale, tmp);
    RowSoft q = p;
    if (drow && more) q = block_softmax(drow, a.C, a.draft_scale, tmp);
    const double ln_sum = row_ln_sum(p);
    const bool broken = p.Z != p.Z || q.Z != q.Z;
    if (more && !broken) {
      const bool in = x < a.C;
      const double px = in ? (double)row_exp(p, (float)row[x]) / (double)p.Z : 0.0;
      double qx = 1.0;
      if (drow) qx = in ? (double)row_exp(q, (float)drow[x]) / (double)q.Z : 0.0;
      if ((double)a.accept_u[r] * qx < px) {
        if (tid == 0) {
          a.tokens[r] = x;
          a.logp[r] = (float)row_logp(p, (float)row[x], a.scale, ln_sum);
        }
        continue;
      }
    }
    // the row that a token is drawn from
    const auto weight = [&](int c, int how) {
      const float pc = row_exp(p, (float)row[c]) / p.Z;
      if (how == 0) return pc;
      const float qc = drow ? row_exp(q, (float)drow[c]) / q.Z : (c == x ? 1.0f : 0.0f);
      return fmaxf(pc - qc, 0.0f);
    };
    int token = -1;
    const double u = a.sample_u[s];
    if (!broken && u == u) {
      int how = more;
      double total = 0.0;
      for (;; how = 0) {
        double sum = 0.0;
        for (int c = tid; c < a.C; c += 256) sum += (double)weight(c, how);
        total = block_sum(sum, tmp);
        if (total > 0.0 || !how) break;
      }
      const double goal = u * total;
      double before = 0.0;
      int last = -1;
      for (int c0 = 0; c0 < a.C && token < 0; c0 += 256) {
        const int c = c0 + tid;
        const float w = c < a.C ? weight(c, how) : 0.0f;
        double upto = w;
        for (int o = 1; o < 64; o *= 2) {
          const double y = __shfl_up(upto, o);
          if ((tid & 63) >= o) upto += y;
        }
        if ((tid & 63) == 63) wave_tot[tid >> 6] = upto;
        if (tid == 0) found = INT32_MAX;
        __syncthreads();
        for (int k = 0; k < (tid >> 6); ++k) upto += wave_tot[k];
        if (c < a.C && before + upto > goal) atomicMin(&found, c);
        if (c < a.C && w > 0.0f) last = c;
        __syncthreads();
        if (found != INT32_MAX) token = found;
        before += wave_tot[0] + wave_tot[1] + wave_tot[2] + wave_tot[3];
        __syncthreads();
      }
      if (token < 0) {               // u of 1 and more
        if (tid == 0) found = -1;
        __syncthreads();
        atomicMax(&found, last);
        __syncthreads();
        token = found;
      }
    }
    if (tid == 0) {
      a.tokens[r] = token;
      a.logp[r] = token >= 0 ? (float)row_logp(p, (float)row[token], a.scale, ln_sum)
                             : (broken ? __builtin_nanf("") : 0.0f);
      a.accepted[s] = (int)(r - lo);
    }
    return;
  }
}

__global__ void verify_clear_kernel(VerifyArgs a) {
  const int64_t r = linear_block() * 256 + threadIdx.x;
  if (r >= a.R) return;
  a.tokens[r] = -1;
  a.logp[r] = 0.0f;
}

template <typename T>
hipError_t verify_t(const VerifyArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(verify_clear_kernel, linear_grid((a.R + 255) / 256), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 0) return e;
  hipLaunchKernelGGL(verify_kernel<T>, linear_grid(a.S), dim3(256), 0, s, a, (const T*)a.z,
                     (const T*)a.d);
  return hipGetLastError();
}

}  // namespace

hipError_t run_verify(const VerifyArgs& a, char* ws, hipStream_t s) {
  if (a.dtype == LIK_F16) return verify_t<_Float16>(a, s);
  if (a.dtype == LIK_BF16) return verify_t<__bf16>(a, s);
  return verify_t<float>(a, s);
}

}  // namespace lik

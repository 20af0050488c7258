// Attention over the 8-bit cache (include/lik_cache.h, lik_cache_attention).
#include <hip/hip_runtime.h>

#include "lik_cache_device.h"
#include "lik_cache_kernels.h"

namespace lik {

namespace {

constexpr float kNegInf = -__builtin_inff();

// One wave per query token and head.
template <typename T>
__global__ __launch_bounds__(64) void attend_kernel(AttendArgs a) {
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, dim = a.dim, bs = a.block_size;
  const int kv = h / (a.q_heads / a.kv_heads);
  int s = -1, at = 0, n = 0;
  for (int i = 0; i < a.S; ++i) {
    int lo = a.q_offsets[i], hi = a.q_offsets[i + 1];
    if (t >= lo && t < hi && s < 0) {
      s = i;
      at = t - lo;
      n = (hi < a.T ? hi : a.T) - lo;
    }
  }
  int seen = 0;
  if (s >= 0) {
    const int64_t most = (int64_t)a.max_blocks * bs;
    int64_t len = a.kv_len[s];
    len = len < 0 ? 0 : (len > most ? most : len);
    const int64_t p = len - n + at + 1;
    seen = p < 0 ? 0 : (int)p;
  }
  const T* q = (const T*)a.q + t * a.q_ld + (int64_t)h * dim;
  float o[4] = {0, 0, 0, 0}, m = kNegInf, l = 0.0f;
  for (int j0 = 0; j0 < seen; j0 += 64) {
    const int j = j0 + lane;
    float score = kNegInf;
    int b = -1;
    if (j < seen) b = a.table[s * a.table_ld + j / bs];
    if (b >= a.num_blocks) b = -1;
    if (b >= 0) {
      const uint8_t* k = a.k.codes + b * a.k.stride + ((int64_t)kv * bs + j % bs) * dim;
      float dot = 0.0f;
      for (int i = 0; i < dim; ++i) dot = fmaf((float)q[i], from_code(k[i]), dot);
      score = dot * clamp_scale(a.k.scale[(int64_t)b * a.kv_heads + kv]) * a.scale;
    }
    const bool nan = __any(score != score);
    const float top = nan ? __builtin_nanf("") : cache_wave_max(fmaxf(score, m));
    if (top == kNegInf) continue;
    const float keep = m == kNegInf ? 0.0f : expf(m - top);
    const float w = b >= 0 ? expf(score - top) : 0.0f;
    float sum = w;
    for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
    l = l * keep + sum;
    m = top;
    for (int i = 0; i < 4; ++i) o[i] *= keep;
    for (int y = 0; y < 64 && j0 + y < seen; ++y) {
      const int by = __shfl(b, y);
      if (by < 0) continue;
      const float wy = __shfl(w, y) * clamp_scale(a.v.scale[(int64_t)by * a.kv_heads + kv]);
      const uint8_t* v = a.v.codes + by * a.v.stride + (int64_t)kv * bs * dim + (j0 + y) % bs;
      for (int i = 0; i * 64 + lane < dim; ++i)
        o[i] = fmaf(wy, from_code(v[(i * 64 + lane) * bs]), o[i]);
    }
  }
  T* out = (T*)a.out + t * a.out_ld + (int64_t)h * dim;
  for (int i = 0; i * 64 + lane < dim; ++i) out[i * 64 + lane] = (T)(m == kNegInf ? 0.0f : o[i] / l);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + h] = m == kNegInf ? m : m + logf(l);
}

}  // namespace

size_t attend_workspace(int64_t T, int64_t S, int64_t q_heads, int64_t kv_heads, int64_t dim,
                        lik_dtype dtype) {
  return 0;
}

hipError_t run_attend(const AttendArgs& a, char* ws, hipStream_t s) {
  const dim3 grid(a.T, a.q_heads);
  if (a.dtype == LIK_F16) hipLaunchKernelGGL(attend_kernel<_Float16>, grid, dim3(64), 0, s, a);
  else if (a.dtype == LIK_BF16) hipLaunchKernelGGL(attend_kernel<__bf16>, grid, dim3(64), 0, s, a);
  else hipLaunchKernelGGL(attend_kernel<float>, grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace lik

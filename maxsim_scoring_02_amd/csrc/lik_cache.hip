// Block tables and writes of the 8-bit cache (include/lik_cache.h).
#include <hip/hip_runtime.h>

#include "lik_cache_device.h"
#include "lik_cache_kernels.h"

namespace lik {

namespace {

// Sum of v over the threads before this one, and over all.
__device__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
  for (int o = 1; o < 64; o *= 2) {
    const int64_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) tmp[wave] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < 16; ++w) {
    if (w < wave) before += tmp[w];
    all += tmp[w];
  }
  *total = all;
  return before + x - v;
}

// One workgroup, request after request.
__global__ __launch_bounds__(1024) void tables_kernel(TablesArgs a) {
  __shared__ int64_t tmp[16];
  const int tid = threadIdx.x, bs = a.block_size, N = a.num_blocks;
  const int64_t most = (int64_t)a.max_blocks * bs;
  const int head = a.state[0], count = a.state[1];
  const int64_t head0 = N > 0 && head > 0 ? head % N : 0;
  const int64_t free_blocks = count < 0 ? 0 : (count > N ? N : count);
  int64_t asked = 0, given = 0, tokens = 0, taken = 0, back = 0;
  for (int s0 = 0; s0 < a.S; s0 += 1024) {
    const int s = s0 + tid;
    int64_t o = 0, n = 0;
    if (s < a.S) {
      o = a.old_len[s];
      n = a.new_len[s];
      o = o < 0 ? 0 : (o > most ? most : o);
      n = n < 0 ? 0 : n;
    }
    const int64_t have = (o + bs - 1) / bs, need = (n + bs - 1) / bs;
    const bool fits = need <= a.max_blocks;
    const int64_t ask = fits && need > have ? need - have : 0;
    const int64_t give = fits && need < have ? have - need : 0;
    const int64_t grown = n > o ? n - o : 0;
    int64_t total;
    const int64_t start = asked + block_scan(ask, tmp, &total);
    asked += total;
    const int64_t rel = given + block_scan(give, tmp, &total);
    given += total;
    const int64_t first = tokens + block_scan(grown, tmp, &total);
    tokens += total;
    const bool ok = fits && (ask == 0 || start + ask <= free_blocks);
    block_scan(ok ? ask : 0, tmp, &total);
    taken += total;
    block_scan(ok ? give : 0, tmp, &total);
    back += total;
    if (s >= a.S) continue;
    int32_t* row = a.table + s * a.table_ld;
    a.granted[s] = (int32_t)(ok ? n : o);
    a.offsets[s] = (int32_t)(first < INT32_MAX ? first : INT32_MAX);
    if (ok) {
      for (int64_t i = have; i < need; ++i) row[i] = a.ring[(head0 + start + i - have) % N];
      for (int64_t i = need; i < have; ++i) {
        if (N > 0) a.ring[(head0 + free_blocks + rel + i - need) % N] = row[i];
        row[i] = -1;
      }
    }
    for (int64_t i = 0; i < grown && first + i < a.T; ++i) {
      const int64_t p = o + i;
      const int b = ok ? row[p / bs] : -1;
      a.slots[first + i] = b >= 0 && b < N ? b * bs + (int)(p % bs) : -1;
    }
  }
  for (int64_t i = tokens + tid; i < a.T; i += 1024) a.slots[i] = -1;
  if (tid == 0) {
    a.offsets[a.S] = (int32_t)(tokens < INT32_MAX ? tokens : INT32_MAX);
    if (N > 0) {
      a.state[0] = (int32_t)((head0 + taken) % N);
      const int64_t now = free_blocks - taken + back;
      a.state[1] = (int32_t)(now > N ? N : now);
    }
  }
}

// One wave per token and head: the first token of a block in the call does the
// block, first its keys, then its values.
template <typename T>
__global__ __launch_bounds__(64) void append_kernel(AppendArgs a) {
  const int t = blockIdx.x, h = blockIdx.y, part = blockIdx.z, lane = threadIdx.x;
  const int bs = a.block_size, dim = a.dim;
  const auto block_of = [&](int i) {
    const int slot = a.slots[i];
    return slot < 0 || slot / bs >= a.num_blocks ? -1 : slot / bs;
  };
  const int b = block_of(t);
  if (b < 0 || (t > 0 && block_of(t - 1) == b)) return;
  const CachePart c = a.part[part];
  const T* x = (const T*)a.x[part] + (int64_t)h * dim;
  uint8_t* codes = c.codes + (int64_t)b * c.stride + (int64_t)h * bs * dim;
  float* scale = c.scale + (int64_t)b * a.heads + h;
  // element i of the token at offset o
  const auto at = [&](int o, int i) { return part ? i * bs + o : o * dim + i; };
  float amax = 0.0f;
  bool fresh = false, broken = false;
  int end = t;
  for (; end < a.T && block_of(end) == b; ++end) {
    fresh |= a.slots[end] % bs == 0;
    for (int i = lane; i < dim; i += 64) {
      const float f = (float)x[end * a.ld[part] + i];
      broken |= !(f - f == 0.0f);
      amax = fmaxf(amax, fabsf(f));
    }
  }
  amax = cache_wave_max(amax);
  broken = __any(broken);
  const float was = *scale;
  float now = scale_of(amax);
  if (!fresh) now = grown_scale(was, now);
  if (broken) now = __builtin_nanf("");
  if (!fresh && now != was && now == now) {
    const float k = clamp_scale(was) / now;
    for (int i = lane; i < bs * dim; i += 64) codes[i] = to_code(from_code(codes[i]) * k);
  }
  __syncthreads();
  const float inv = now == now ? 1.0f / now : 0.0f;
  for (int j = t; j < end; ++j)
    for (int i = lane; i < dim; i += 64) {
      const float f = (float)x[j * a.ld[part] + i];
      codes[at(a.slots[j] % bs, i)] = to_code(f - f == 0.0f && inv > 0.0f ? f * inv : 0.0f);
    }
  if (lane == 0) *scale = now;
}

}  // namespace

hipError_t run_tables(const TablesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(tables_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t run_append(const AppendArgs& a, hipStream_t s) {
  const dim3 grid(a.T, a.heads, 2);
  if (a.dtype == LIK_F16) hipLaunchKernelGGL(append_kernel<_Float16>, grid, dim3(64), 0, s, a);
  else if (a.dtype == LIK_BF16) hipLaunchKernelGGL(append_kernel<__bf16>, grid, dim3(64), 0, s, a);
  else hipLaunchKernelGGL(append_kernel<float>, grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace lik

// Block tables and writes of the 8-bit cache (include/lik_cache.h).
#include <hip/hip_runtime.h>

#include "lik_cache_device.h"
#include "lik_cache_kernels.h"

namespace lik {

namespace {

// ---------------------------------------------------------------------------
// block tables
// ---------------------------------------------------------------------------

// What a request asks for.
struct Change {
  int old_len, new_len;
  int have, need;                        // blocks
  bool fits;
  __device__ __forceinline__ int ask() const { return fits && need > have ? need - have : 0; }
  __device__ __forceinline__ int give() const { return fits && need < have ? have - need : 0; }
  __device__ __forceinline__ int grown() const {
    return new_len > old_len ? new_len - old_len : 0;
  }
};
__device__ __forceinline__ Change change_of(const TablesArgs& a, int s, int shift) {
  const int most = (int)((uint32_t)a.max_blocks << shift);
  const int o = a.old_len[s], n = a.new_len[s], round = (1 << shift) - 1;
  Change c;
  c.old_len = o < 0 ? 0 : (o > most ? most : o);
  c.new_len = n < 0 ? 0 : n;
  c.have = (int)(((uint32_t)c.old_len + round) >> shift);
  c.need = (int)(((uint32_t)c.new_len + round) >> shift);
  c.fits = c.need <= a.max_blocks;
  return c;
}

constexpr int kTablesThreads = 256;

// Three running sums over a workgroup: before this thread, and of all.
struct Sums {
  int64_t ask, give, grown;
};
struct ScanLds {
  Sums wave[kTablesThreads / 64];
};
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int64_t y = __shfl_up(v, o);
    if ((threadIdx.x & 63) >= (unsigned)o) v += y;
  }
  return v;
}
__device__ __forceinline__ Sums scan3(Sums v, ScanLds& lds, Sums* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Sums x{wave_scan(v.ask), wave_scan(v.give), wave_scan(v.grown)};
  __syncthreads();
  if (lane == 63) lds.wave[wave] = x;
  __syncthreads();
  x.ask -= v.ask;
  x.give -= v.give;
  x.grown -= v.grown;
  *all = Sums{0, 0, 0};
  for (int w = 0; w < kTablesThreads / 64; ++w) {
    const Sums y = lds.wave[w];
    if (w < wave) {
      x.ask += y.ask;
      x.give += y.give;
      x.grown += y.grown;
    }
    all->ask += y.ask;
    all->give += y.give;
    all->grown += y.grown;
  }
  return x;
}

__device__ __forceinline__ int clamp_int(int64_t x) { return x < INT32_MAX ? (int)x : INT32_MAX; }

// The last of n entries of a rising array that is at most x; the first is.
__device__ __forceinline__ int last_at_most(const int64_t* v, int64_t x) {
  int b = 0;
#pragma unroll
  for (int step = kTablesThreads / 2; step > 0; step /= 2)
    if (v[b + step] <= x) b += step;
  return b;
}

// A place in the ring; a consistent pool goes round its end once at most.
__device__ __forceinline__ int ring_at(int64_t i, int N) {
  if (i >= N) i -= N;
  return (int)(i < N ? i : i % N);
}

// One launch.  Workgroup (x, y) takes the requests 256 x .. 256 x + 255 (and further
// ones, gridDim.x * 256 apart), and of their table entries and slots every
// gridDim.y-th 256: it sums what all requests before ask for by itself, which is a
// few loads a thread for as many requests as a batch has, and needs no workgroup to
// wait for another.  The workgroup that is last to have read the pool's state
// (counted in ring_state[2], which it sets back) moves it.  Blocks to take and room
// for blocks given back lie apart in the ring, so entries are independent.
// 64 requests, 100000 slots: see the table of cases.
__global__ __launch_bounds__(kTablesThreads) void tables_kernel(TablesArgs a) {
  __shared__ ScanLds lds;
  __shared__ int64_t entry0[kTablesThreads], token0[kTablesThreads];
  __shared__ int s_old[kTablesThreads], s_have[kTablesThreads], s_need[kTablesThreads];
  __shared__ int64_t s_ring[kTablesThreads];     // where its blocks come from or go to; -1: not granted
  __shared__ int is_last, s_state[2];
  const int tid = threadIdx.x, bs = a.block_size, N = a.num_blocks;
  const int shift = __builtin_ctz(bs);
  // one thread reads the state, and counts once it has it
  if (tid == 0) {
    const int h = a.state[0], f = a.state[1], n = (int)(gridDim.x * gridDim.y);
    s_state[0] = N > 0 && h > 0 ? h % N : 0;
    s_state[1] = f < 0 ? 0 : (f > N ? N : f);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    is_last = n == 1 || atomicAdd(&a.state[2], 1) == n - 1;
  }
  __syncthreads();
  const int head = s_state[0], free_blocks = s_state[1];

  Sums upto{0, 0, 0};                            // of all requests before s0
  int64_t tokens = 0, taken = 0, back = 0;
  bool whole = false;                            // taken and back are those of all
  const auto ok_of = [&](const Change& c, int64_t before) {
    return c.fits && (c.ask() == 0 || before + c.ask() <= free_blocks);
  };
  int done = 0;
  for (int s0 = blockIdx.x * kTablesThreads; s0 < a.S || done == 0;
       s0 += gridDim.x * kTablesThreads) {
    // sums of the requests between
    Sums mine{0, 0, 0}, all;
    for (int s = done + tid; s < s0 && s < a.S; s += kTablesThreads) {
      const Change c = change_of(a, s, shift);
      mine.ask += c.ask();
      mine.give += c.give();
      mine.grown += c.grown();
    }
    scan3(mine, lds, &all);
    upto.ask += all.ask;
    upto.give += all.give;
    upto.grown += all.grown;
    if (s0 >= a.S) break;

    const int s = s0 + tid;
    Change c{0, 0, 0, 0, false};
    if (s < a.S) c = change_of(a, s, shift);
    const Sums before = scan3(Sums{c.ask(), c.give(), c.grown()}, lds, &all);
    const int64_t start = upto.ask + before.ask, rel = upto.give + before.give;
    const bool ok = ok_of(c, start);
    const int64_t first = upto.grown + before.grown;
    const int moves = ok ? c.ask() + c.give() : 0;
    Sums moved;
    const Sums entry = scan3(Sums{moves, 0, 0}, lds, &moved);
    entry0[tid] = entry.ask;
    token0[tid] = before.grown;
    s_old[tid] = c.old_len;
    s_have[tid] = c.have;
    s_need[tid] = c.need;
    s_ring[tid] = !ok ? -1 : (c.ask() ? head + start : (int64_t)head + free_blocks + rel);
    if (s < a.S && blockIdx.y == 0) {
      a.granted[s] = ok ? c.new_len : c.old_len;
      a.offsets[s] = clamp_int(first);
    }
    __syncthreads();
    // table entries
    const int64_t step = (int64_t)gridDim.y * kTablesThreads;
    for (int64_t e = (int64_t)blockIdx.y * kTablesThreads + tid; e < moved.ask; e += step) {
      const int i = last_at_most(entry0, e);
      const int k = (int)(e - entry0[i]);
      int32_t* row = a.table + (s0 + i) * a.table_ld;
      // a request without blocks granted has no ring to look at: N > 0 where it takes some
      if (s_need[i] > s_have[i]) {
        row[s_have[i] + k] = a.ring[ring_at(s_ring[i] + k, N)];
      } else {
        if (N > 0) a.ring[ring_at(s_ring[i] + k, N)] = row[s_need[i] + k];
        row[s_need[i] + k] = -1;
      }
    }
    // slots
    const int64_t most = a.T - upto.grown, here = all.grown < most ? all.grown : most;
    for (int64_t e = (int64_t)blockIdx.y * kTablesThreads + tid; e < here; e += step) {
      const int i = last_at_most(token0, e);
      const int p = s_old[i] + (int)(e - token0[i]);
      int b = -1;
      if (s_ring[i] >= 0) {
        const int at = p >> shift;
        b = at < s_have[i] ? a.table[(s0 + i) * a.table_ld + at]
                           : a.ring[ring_at(s_ring[i] + at - s_have[i], N)];
      }
      a.slots[upto.grown + e] = (unsigned)b < (unsigned)N ? (b << shift) + (p & (bs - 1)) : -1;
    }
    upto.ask += all.ask;
    upto.give += all.give;
    upto.grown += all.grown;
    done = s0 + kTablesThreads;
    if (gridDim.x == 1) {
      Sums x;
      scan3(Sums{ok ? c.ask() : 0, ok ? c.give() : 0, 0}, lds, &x);
      taken += x.ask;
      back += x.give;
      whole = true;
    }
    __syncthreads();
  }
  // tokens of the requests behind, then what no request has
  {
    Sums mine{0, 0, 0}, all;
    for (int s = done + tid; s < a.S; s += kTablesThreads) mine.grown += change_of(a, s, shift).grown();
    scan3(mine, lds, &all);
    tokens = upto.grown + all.grown;
  }
  const int64_t linear = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t threads = (int64_t)gridDim.x * gridDim.y * kTablesThreads;
  for (int64_t i = tokens + linear * kTablesThreads + tid; i < a.T; i += threads) a.slots[i] = -1;
  if (linear == 0 && tid == 0) a.offsets[a.S] = clamp_int(tokens);
  if (!is_last) return;
  if (!whole) {
    Sums sum{0, 0, 0};
    for (int s0 = 0; s0 < a.S; s0 += kTablesThreads) {
      Change c{0, 0, 0, 0, false};
      if (s0 + tid < a.S) c = change_of(a, s0 + tid, shift);
      Sums all, x;
      const Sums before = scan3(Sums{c.ask(), 0, 0}, lds, &all);
      const bool ok = ok_of(c, sum.ask + before.ask);
      scan3(Sums{ok ? c.ask() : 0, ok ? c.give() : 0, 0}, lds, &x);
      sum.ask += all.ask;
      taken += x.ask;
      back += x.give;
    }
  }
  if (tid == 0 && N > 0) {
    const int64_t now = free_blocks - taken + back;
    a.state[0] = (int)((head + taken) % N);
    a.state[1] = (int)(now > N ? N : now);
  }
  if (tid == 0) a.state[2] = 0;
}

// ---------------------------------------------------------------------------
// appends
// ---------------------------------------------------------------------------

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
  // workgroups for the requests, and so many times them that a thread has about 16
  // slots or, where few are asked for, table entries
  const int64_t x = a.S < 256 * kTablesThreads ? (a.S + kTablesThreads - 1) / kTablesThreads : 256;
  const int64_t groups = x > 0 ? x : 1;
  int64_t y = ((int64_t)a.T + groups * 4096 - 1) / (groups * 4096);
  const int64_t most = 1024 / groups > 1 ? 1024 / groups : 1;
  y = y < 1 ? 1 : (y > most ? most : y);
  hipLaunchKernelGGL(tables_kernel, dim3((unsigned)groups, (unsigned)y), dim3(kTablesThreads), 0, s,
                     a);
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

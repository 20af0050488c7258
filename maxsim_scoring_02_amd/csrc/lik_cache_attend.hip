// Attention over the 8-bit cache (include/lik_cache.h, lik_cache_attention).
//
//   out_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j),  j <= pos(i)
//
// The rows of a request and a head of the cache are its query tokens times the
// query heads that share the head; 16 * MT of them are a row tile.  A wave takes a
// row tile over a range of the cache, 64 tokens at a time, alone: the scores
// S^T = K Q^T and the sums O^T = V^T P^T run on v_mfma_f32_16x16x32_f16, where an
// 8-bit code is exact as float16, and their operands come from memory straight into
// registers.
//
// * Lane 16 j + c has query row c and the 16 tokens 16 j .. 16 j + 15 of a tile,
//   which lie in one block: its scale is one number a lane.  The key's goes into the
//   factor of the score, the value's into the exponent:
//     w' = 2^(score log2(e) + log2(v_scale) - m),   P = w',   sum w = sum w' / v_scale
//   so that P is at most 2^8 and float16 whatever the scales are, and neither costs
//   an instruction per score.
// * The tokens of a score tile are chosen so that its output registers are the
//   next product's operand: no weight crosses a lane.
// * Values lie dim by dim in the cache, so 16 tokens of one dim are a 16-byte load
//   and the operand of two products.
// * The maximum m moves only when a score passes it by 2^8.
//
// The work of a head is numbered (request, row tile, 64 tokens) and cut into
// equal ranges, one a wave, whatever the lengths are.  A row tile that lies in
// several ranges leaves its sums in the workspace, and a second kernel merges them.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lik_cache_device.h"
#include "lik_cache_kernels.h"

namespace lik {

namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;                // tokens
constexpr float kNegInf = -__builtin_inff();
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// x and its partner 16 or 32 lanes away
template <bool Wide>
__device__ __forceinline__ void pair_of(float x, float* a, float* b) {
  const uint32_t u = __float_as_uint(x);
  const auto r = Wide ? __builtin_amdgcn_permlane32_swap(u, u, false, false)
                      : __builtin_amdgcn_permlane16_swap(u, u, false, false);
  *a = __uint_as_float(r[0]);
  *b = __uint_as_float(r[1]);
}
// Over the four lanes of a query row; every lane gets the result.
__device__ __forceinline__ float row_max4(float x) {
  float a, b;
  pair_of<false>(x, &a, &b);
  pair_of<true>(fmaxf(a, b), &a, &b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float row_sum4(float x) {
  float a, b;
  pair_of<false>(x, &a, &b);
  pair_of<true>(a + b, &a, &b);
  return a + b;
}

// Eight codes (two words) as float16.
__device__ __forceinline__ half8 widen(uint32_t lo, uint32_t hi) {
  half8 h;
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  h[0] = a[0]; h[1] = a[1]; h[2] = b[0]; h[3] = b[1];
  h[4] = c[0]; h[5] = c[1]; h[6] = d[0]; h[7] = d[1];
  return h;
}

__device__ __forceinline__ f32x4 mma(half8 a, half8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// What a launch knows of the work: workers (waves) a head, rows a tile.
struct Split {
  int workers;
  int least;                             // fewest tiles a range
};

// One request.
struct Request {
  int q0, n, len, rows, row_tiles, kv_tiles;
};
template <int M>
__device__ __forceinline__ Request request_of(const AttendArgs& a, int s) {
  Request r;
  const int lo = a.q_offsets[s], hi = a.q_offsets[s + 1];
  r.q0 = lo < 0 ? 0 : (lo > a.T ? a.T : lo);
  const int end = hi > a.T ? a.T : hi;
  r.n = end > r.q0 ? end - r.q0 : 0;
  const int64_t most = a.num_blocks > 0 ? (int64_t)a.max_blocks * a.block_size : 0;
  const int len = a.kv_len[s];
  r.len = len < 0 ? 0 : (len > most ? (int)most : len);
  r.rows = r.n * (a.q_heads / a.kv_heads);
  r.row_tiles = (r.rows + M - 1) / M;
  r.kv_tiles = r.len > 0 ? (int)(((int64_t)r.len + kTile - 1) / kTile) : 1;
  return r;
}

// The numbering of a head's work, found by the 256 threads of a workgroup: sums
// over buckets of requests, and the range of a worker.
struct Plan {
  int64_t total, chunk;
  int per;                               // requests a bucket
  const int64_t* before;                 // [257] units before each bucket, in LDS
};
template <int M>
__device__ __forceinline__ Plan make_plan(const AttendArgs& a, const Split& sp, int64_t* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Plan p;
  p.per = (a.S + 255) / 256;
  int64_t units = 0;
  const int first = tid * p.per, last = first + p.per < a.S ? first + p.per : a.S;
  for (int s = first; s < last; ++s) {
    const Request r = request_of<M>(a, s);
    units += (int64_t)r.row_tiles * r.kv_tiles;
  }
  int64_t x = units;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int64_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) lds[257 + wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += lds[257 + w];
  lds[tid + 1] = x;
  if (tid == 0) lds[0] = 0;
  __syncthreads();
  p.before = lds;
  p.total = lds[256];
  p.chunk = (p.total + sp.workers - 1) / sp.workers;
  if (p.chunk < sp.least) p.chunk = sp.least;
  return p;
}

// The request that holds unit u, and the units before it.
template <int M>
__device__ __forceinline__ void find_unit(const AttendArgs& a, const Plan& p, int64_t u, int* s,
                                          int64_t* pos, Request* r) {
  int b = 0;
#pragma unroll
  for (int step = 128; step > 0; step /= 2)
    if (p.before[b + step] <= u) b += step;
  *s = b * p.per;
  *pos = p.before[b];
  for (;; ++*s) {
    *r = request_of<M>(a, *s);
    const int64_t units = (int64_t)r->row_tiles * r->kv_tiles;
    if (u < *pos + units || *s + 1 >= a.S) return;
    *pos += units;
  }
}

// Positions that a row of a request attends to.
__device__ __forceinline__ int seen_of(const Request& r, int row, int group) {
  const int p = r.len - r.n + row / group + 1;
  return p < 0 ? 0 : (p > r.len ? r.len : p);
}
// Tiles of 64 tokens that row tile t needs, one at least.
template <int M>
__device__ __forceinline__ int tiles_of(const Request& r, int t, int group) {
  const int end = (t + 1) * M < r.rows ? (t + 1) * M : r.rows;
  const int seen = seen_of(r, end - 1, group);
  return seen > 0 ? (seen + kTile - 1) / kTile : 1;
}

// Partial sums in the workspace: [head][worker][2] row tiles of M rows.
struct Partial {
  float* o;                              // [M][D]
  float2* ml;                            // [M]: m, l
};
template <int M, int D>
__device__ __forceinline__ Partial partial_at(char* ws, const AttendArgs& a, const Split& sp,
                                              int head, int64_t worker, int slot) {
  const int64_t n = (int64_t)a.kv_heads * sp.workers * 2;
  const int64_t i = ((int64_t)head * sp.workers + worker) * 2 + slot;
  return {(float*)ws + i * M * D, (float2*)((float*)ws + n * M * D) + i * M};
}

template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  *(t4*)p = t4{(T)a, (T)b, (T)c, (T)d};
}

// A row tile over tiles kt0 .. kt1 - 1.
template <typename T, int D, int MT>
struct RowTile {
  static constexpr bool kTwo = std::is_same<T, float>::value;   // float32: two float16 parts
  static constexpr int kParts = kTwo ? 2 : 1;
  static constexpr int M = 16 * MT, NC = D / 32, NI = D / 64, ND = D / 16;
  // how far a score may pass the maximum before it moves (float32's parts: not at all)
  static constexpr float kSlack = kTwo ? 0.0f : 8.0f;

  half8 q[kParts][MT][NC];
  float factor[MT];                      // scale log2(e) 2^-k of the lane's query row
  int seen[MT];
  float m[MT], l[MT];
  f32x4 o[MT][ND];

  __device__ __forceinline__ void load_queries(const AttendArgs& a, const Request& r, int t,
                                               int head, int lane) {
    const int group = a.q_heads / a.kv_heads, c = lane & 15, j = lane >> 4;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = t * M + mt * 16 + c;
      const bool there = row < r.rows;
      const int token = there ? row / group : 0, h = there ? row - token * group : 0;
      seen[mt] = there ? seen_of(r, row, group) : 0;
      const T* x = (const T*)a.q + (int64_t)(r.q0 + token) * a.q_ld +
                   (int64_t)(head * group + h) * D;
      float f[NC][8], top = 0.0f;
      bool broken = false;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        typedef T t8 __attribute__((ext_vector_type(8), aligned(16)));
        const t8 v = *(const t8*)(x + (i >> 1) * 64 + j * 16 + (i & 1) * 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[i][e] = (float)v[e];
          top = fmaxf(top, fabsf(f[i][e]));
          broken |= !(f[i][e] - f[i][e] == 0.0f);
        }
      }
      top = row_max4(top);
      broken = row_max4(broken ? 1.0f : 0.0f) > 0.0f;
      // the row's largest number to [2^14, 2^15): exact, and small ones keep their digits
      const int k = top > 0.0f && !broken ? 14 - ilogbf(top) : 0;
      factor[mt] = broken ? __builtin_nanf("") : ldexpf(a.scale * kLog2e, -k);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = broken ? 0.0f : ldexpf(f[i][e], k);
          q[0][mt][i][e] = (_Float16)y;
          if constexpr (kTwo) q[kParts - 1][mt][i][e] = (_Float16)(y - (float)(_Float16)y);
        }
      }
      m[mt] = kNegInf;
      l[mt] = 0.0f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[mt][d] = f32x4{0, 0, 0, 0};
    }
  }

  __device__ __forceinline__ void run(const AttendArgs& a, int s, int len, int head, int kt0,
                                      int kt1, int open, int lane) {
    const int c = lane & 15, j = lane >> 4, bs = a.block_size;
    const int shift = __builtin_ctz(bs);
    const int32_t* table = a.table + (int64_t)s * a.table_ld;
    const uint8_t* kb = a.k.codes + (int64_t)head * bs * D + j * 16;
    const uint8_t* vb = a.v.codes + ((int64_t)head * D + c) * bs;
    for (int kt = kt0; kt < kt1; ++kt) {
      const int base = kt * kTile;
      // the lane's own block (16 j), and that of the key row it loads (4 rows each)
      const int tj = base + j * 16, tk = base + (c >> 2) * 16;
      int bj = tj < len ? table[tj >> shift] : -1;
      int bk = tk < len ? table[tk >> shift] : -1;
      const bool there = (unsigned)bj < (unsigned)a.num_blocks;
      if (!there) bj = 0;
      if ((unsigned)bk >= (unsigned)a.num_blocks) bk = 0;
      const uint8_t* kp = kb + (int64_t)bk * a.k.stride + ((tk & (bs - 1)) + (c & 3)) * D;
      const uint8_t* vp = vb + (int64_t)bj * a.v.stride + (tj & (bs - 1));
      u32x4 kr[4][NI], vr[ND];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int i = 0; i < NI; ++i) kr[tt][i] = *(const u32x4*)(kp + tt * 4 * D + i * 64);
#pragma unroll
      for (int d = 0; d < ND; ++d) vr[d] = *(const u32x4*)(vp + d * 16 * bs);
      float ks = clamp_scale(a.k.scale[(int64_t)bj * a.kv_heads + head]);
      float vs = clamp_scale(a.v.scale[(int64_t)bj * a.kv_heads + head]);
      const bool no_keys = there && ks != ks, no_values = there && vs != vs;
      if (ks != ks) ks = 1.0f;
      if (vs != vs) vs = 1.0f;
      const float lv = __builtin_amdgcn_logf(vs), iv = __builtin_amdgcn_rcpf(vs);

      f32x4 sc[MT][4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) sc[mt][tt] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const half8 k8 = widen(kr[tt][i >> 1][(i & 1) * 2], kr[tt][i >> 1][(i & 1) * 2 + 1]);
#pragma unroll
          for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) sc[mt][tt] = mma(k8, q[part][mt][i], sc[mt][tt]);
        }
      }
      // tokens behind a row's own, behind the length, or in no block
      const bool all = __all(there) && base + kTile <= open;
      if (!all) {
        const int valid = there ? len - tj : 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int lim = there ? seen[mt] - tj : 0;
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (tt * 4 + e >= lim) sc[mt][tt][e] = kNegInf;
        }
        // codes of what is not there may be no numbers: 0
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int left = valid - w * 4;
            const uint32_t mask = left >= 4 ? ~0u : (left <= 0 ? 0u : (1u << (left * 8)) - 1u);
            vr[d][w] &= mask;
          }
      }
      // a block that is NaN makes NaN what is attended to, and nothing else
      if (__any(no_keys || no_values)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          bool sees = false;
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sees |= sc[mt][tt][e] != kNegInf;
              if (no_keys && sc[mt][tt][e] != kNegInf) sc[mt][tt][e] = __builtin_nanf("");
            }
          if (row_max4(sees && no_values ? 1.0f : 0.0f) > 0.0f)
#pragma unroll
            for (int d = 0; d < ND; ++d) o[mt][d] = o[mt][d] * __builtin_nanf("");
        }
      }
      half8 p[kParts][MT][2];
      float want[MT];
      bool moves = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float top = fmaxf(fmaxf(sc[mt][0][0], sc[mt][0][1]), fmaxf(sc[mt][0][2], sc[mt][0][3]));
#pragma unroll
        for (int tt = 1; tt < 4; ++tt)
          top = fmaxf(top, fmaxf(fmaxf(sc[mt][tt][0], sc[mt][tt][1]),
                                 fmaxf(sc[mt][tt][2], sc[mt][tt][3])));
        float cf = factor[mt] * ks;
        if (cf < 0x1p-126f) cf = 0x1p-126f;          // -inf * 0 would be NaN
        want[mt] = row_max4(fmaf(top, cf, lv));
        moves |= want[mt] > m[mt] + kSlack;
      }
      if (__any(moves)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float now = fmaxf(m[mt], want[mt]);
          const float keep = m[mt] == kNegInf ? 0.0f : exp2_fast(m[mt] - now);
          m[mt] = now;
          l[mt] *= keep;
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][d][e] *= keep;
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float cf = factor[mt] * ks;
        if (cf < 0x1p-126f) cf = 0x1p-126f;
        float shiftv = lv - (m[mt] == kNegInf ? 0.0f : m[mt]);
        // The product below is exact and m is rounded: they are apart by up to 2^-24 |m|.
        // Where that is much the scores are rounded first, as m was.
        if (__any(fabsf(m[mt]) > 0x1p26f && m[mt] != kNegInf)) {
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (sc[mt][tt][e] != kNegInf)
                sc[mt][tt][e] = fmaf(sc[mt][tt][e], cf, lv) - (m[mt] == kNegInf ? 0.0f : m[mt]);
          cf = 1.0f;
          shiftv = 0.0f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = exp2_fast(fmaf(sc[mt][tt][e], cf, shiftv));
            sum += w;
            p[0][mt][tt >> 1][(tt & 1) * 4 + e] = (_Float16)w;
            if constexpr (kTwo)
              p[kParts - 1][mt][tt >> 1][(tt & 1) * 4 + e] = (_Float16)(w - (float)(_Float16)w);
          }
        }
        l[mt] = fmaf(sum, iv, l[mt]);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const half8 v8 = widen(vr[d][half * 2], vr[d][half * 2 + 1]);
#pragma unroll
          for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][d] = mma(v8, p[part][mt][half], o[mt][d]);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) l[mt] = row_sum4(l[mt]);
  }

  __device__ __forceinline__ void finish(const AttendArgs& a, const Request& r, int t, int head,
                                         int lane) const {
    const int group = a.q_heads / a.kv_heads, c = lane & 15, j = lane >> 4;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = t * M + mt * 16 + c;
      if (row >= r.rows) continue;
      const int token = row / group, h = head * group + row - token * group;
      const float inv = l[mt] == 0.0f ? 0.0f : 1.0f / l[mt];
      T* out = (T*)a.out + (int64_t)(r.q0 + token) * a.out_ld + (int64_t)h * D + j * 4;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        store4(out + d * 16, o[mt][d][0] * inv, o[mt][d][1] * inv, o[mt][d][2] * inv,
               o[mt][d][3] * inv);
      if (a.lse && j == 0)
        a.lse[(int64_t)(r.q0 + token) * a.q_heads + h] =
            l[mt] == 0.0f ? kNegInf : (float)(kLn2 * ((double)m[mt] + log2((double)l[mt])));
    }
  }

  __device__ __forceinline__ void save(const Partial& p, const Request& r, int t, int lane) const {
    const int c = lane & 15, j = lane >> 4;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int i = mt * 16 + c;
      if (t * M + i >= r.rows) continue;
#pragma unroll
      for (int d = 0; d < ND; ++d) *(f32x4*)(p.o + i * D + d * 16 + j * 4) = o[mt][d];
      if (j == 0) p.ml[i] = make_float2(m[mt], l[mt]);
    }
  }
};

// Rows outside every request.
template <typename T>
__device__ __forceinline__ void clear_outside(const AttendArgs& a, int64_t thread,
                                              int64_t threads) {
  int lo = a.S > 0 ? a.q_offsets[0] : 0, hi = a.S > 0 ? a.q_offsets[a.S] : 0;
  lo = lo < 0 ? 0 : (lo > a.T ? a.T : lo);
  hi = hi < lo ? lo : (hi > a.T ? a.T : hi);
  const int64_t outside = (int64_t)a.T - (hi - lo), width = (int64_t)a.q_heads * a.dim;
  if (outside == 0) return;
  for (int64_t i = thread; i < outside * width / 8; i += threads) {
    int64_t t = i * 8 / width;
    const int64_t x = i * 8 - t * width;
    if (t >= lo) t += hi - lo;
    T* out = (T*)a.out + t * a.out_ld + x;
    store4(out, 0, 0, 0, 0);
    store4(out + 4, 0, 0, 0, 0);
    if (a.lse && x % a.dim == 0) a.lse[t * a.q_heads + x / a.dim] = kNegInf;
  }
}

template <typename T, int D, int MT>
__global__ __launch_bounds__(256, 2) void attend_kernel(AttendArgs a, Split sp, char* ws) {
  constexpr int M = 16 * MT;
  __shared__ int64_t lds[261];
  const int head = blockIdx.x % a.kv_heads, lane = threadIdx.x & 63;
  clear_outside<T>(a, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
  if (a.S == 0) return;
  const Plan plan = make_plan<M>(a, sp, lds);
  const int64_t worker = (int64_t)(blockIdx.x / a.kv_heads) * 4 +
                         __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int64_t u = worker * plan.chunk;
  const int64_t u0 = u, u1 = u + plan.chunk < plan.total ? u + plan.chunk : plan.total;
  if (u >= u1) return;
  const int group = a.q_heads / a.kv_heads;
  int s;
  int64_t pos;
  Request r;
  find_unit<M>(a, plan, u, &s, &pos, &r);
  while (u < u1) {
    const int64_t units = (int64_t)r.row_tiles * r.kv_tiles;
    if (u >= pos + units) {
      pos += units;
      if (++s >= a.S) return;
      r = request_of<M>(a, s);
      continue;
    }
    const int t = (int)((u - pos) / r.kv_tiles);
    const int64_t first = pos + (int64_t)t * r.kv_tiles;
    const int need = tiles_of<M>(r, t, group);
    const int64_t end = first + r.kv_tiles < u1 ? first + r.kv_tiles : u1;
    const int kt0 = (int)(u - first), kt1 = (int)(end - first < need ? end - first : need);
    if (kt0 < kt1) {
      RowTile<T, D, MT> tile;
      tile.load_queries(a, r, t, head, lane);
      const int seen0 = seen_of(r, t * M, group);
      if (r.len > 0) tile.run(a, s, r.len, head, kt0, kt1, seen0, lane);
      if (kt0 == 0 && kt1 == need) tile.finish(a, r, t, head, lane);
      else tile.save(partial_at<M, D>(ws, a, sp, head, worker, u > u0), r, t, lane);
    }
    u = end;
  }
}

// Merges the row tile that begins in a worker's range and ends in a later one's.
// One workgroup per head and worker; most have none.
template <typename T, int D, int MT>
__global__ __launch_bounds__(256) void merge_kernel(AttendArgs a, Split sp, char* ws) {
  constexpr int M = 16 * MT, L = D / 4;          // L lanes a row
  __shared__ int64_t lds[261];
  const int head = blockIdx.x % a.kv_heads;
  const Plan plan = make_plan<M>(a, sp, lds);
  const int64_t worker = blockIdx.x / a.kv_heads, u0 = worker * plan.chunk;
  const int64_t u1 = u0 + plan.chunk;
  if (u1 >= plan.total) return;
  const int group = a.q_heads / a.kv_heads;
  int s;
  int64_t pos;
  Request r;
  find_unit<M>(a, plan, u1 - 1, &s, &pos, &r);
  const int t = (int)((u1 - 1 - pos) / r.kv_tiles);
  const int64_t first = pos + (int64_t)t * r.kv_tiles;
  const int64_t end = first + tiles_of<M>(r, t, group);
  if (first < u0 || end <= u1) return;
  const int64_t last = (end - 1) / plan.chunk;
  const int rows = r.rows - t * M < M ? r.rows - t * M : M;
  const Partial p0 = partial_at<M, D>(ws, a, sp, head, worker, first > u0);
  for (int i = threadIdx.x / L; i < rows; i += 256 / L) {
    const int d = threadIdx.x % L * 4;
    float m = p0.ml[i].x;
    for (int64_t w = worker + 1; w <= last; ++w)
      m = fmaxf(m, partial_at<M, D>(ws, a, sp, head, w, 0).ml[i].x);
    const float ref = m == kNegInf ? 0.0f : m;
    float k = exp2_fast(p0.ml[i].x - ref), l = p0.ml[i].y * k;
    f32x4 o = *(const f32x4*)(p0.o + i * D + d) * k;
#pragma unroll 4
    for (int64_t w = worker + 1; w <= last; ++w) {
      const Partial p = partial_at<M, D>(ws, a, sp, head, w, 0);
      const float2 ml = p.ml[i];
      k = exp2_fast(ml.x - ref);
      l = fmaf(ml.y, k, l);
      o += *(const f32x4*)(p.o + i * D + d) * k;
    }
    const int row = t * M + i, token = row / group, h = head * group + row - token * group;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    store4((T*)a.out + (int64_t)(r.q0 + token) * a.out_ld + (int64_t)h * D + d, o[0] * inv,
           o[1] * inv, o[2] * inv, o[3] * inv);
    if (a.lse && d == 0)
      a.lse[(int64_t)(r.q0 + token) * a.q_heads + h] =
          l == 0.0f ? kNegInf : (float)(kLn2 * ((double)m + log2((double)l)));
  }
}

int row_tiles_of(int64_t T, int64_t S, int64_t group) {
  return S > 0 && T * group <= 16 * S ? 1 : 2;
}
Split split_of(int64_t kv_heads) {
  constexpr int kWaves = 2048;           // eight a CU
  int64_t w = (kWaves / 4 + kv_heads - 1) / kv_heads * 4;
  return {(int)w, 1};
}

template <typename T, int D, int MT>
hipError_t attend_t(const AttendArgs& a, char* ws, hipStream_t s) {
  const Split sp = split_of(a.kv_heads);
  hipLaunchKernelGGL((attend_kernel<T, D, MT>), dim3(sp.workers / 4 * a.kv_heads), dim3(256), 0, s,
                     a, sp, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 0) return e;
  hipLaunchKernelGGL((merge_kernel<T, D, MT>), dim3(sp.workers * a.kv_heads), dim3(256), 0, s, a,
                     sp, ws);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t attend_d(const AttendArgs& a, char* ws, hipStream_t s) {
  if (row_tiles_of(a.T, a.S, a.q_heads / a.kv_heads) == 1) return attend_t<T, D, 1>(a, ws, s);
  return attend_t<T, D, 2>(a, ws, s);
}

template <typename T>
hipError_t attend_type(const AttendArgs& a, char* ws, hipStream_t s) {
  if (a.dim == 64) return attend_d<T, 64>(a, ws, s);
  if (a.dim == 128) return attend_d<T, 128>(a, ws, s);
  return attend_d<T, 256>(a, ws, s);
}

}  // namespace

size_t attend_workspace(int64_t T, int64_t S, int64_t q_heads, int64_t kv_heads, int64_t dim,
                        lik_dtype dtype) {
  if (S == 0) return 0;
  const int64_t M = 16 * row_tiles_of(T, S, q_heads / kv_heads);
  return (size_t)(kv_heads * split_of(kv_heads).workers * 2 * M * (dim + 2) * 4);
}

hipError_t run_attend(const AttendArgs& a, char* ws, hipStream_t s) {
  if (a.dtype == LIK_F16) return attend_type<_Float16>(a, ws, s);
  if (a.dtype == LIK_BF16) return attend_type<__bf16>(a, ws, s);
  return attend_type<float>(a, ws, s);
}

}  // namespace lik

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
//   so that P is float16 with the largest of a row near float16's end whatever the scales
//   are, and neither costs an instruction per score.
// * The tokens of a score tile are chosen so that its output registers are the
//   next product's operand: no weight crosses a lane.
// * Values lie dim by dim in the cache, so 16 tokens of one dim are a 16-byte load
//   and the operand of two products.
// * The reference m moves only when a weight would leave float16's range (RowTile).
//
// The work of a head is numbered (request, row tile, 64 tokens of the request's length)
// and cut into equal ranges, one a wave.  What lies behind a row tile's own positions is
// numbered too and not done: nothing of it in single tokens and drafts, an eighth in
// prompts behind long caches, half where nothing was cached before, where the busiest
// waves have twice the mean.  A row tile that lies in several ranges leaves its sums
// in the workspace, and a second kernel merges them.
//
// 64 requests of 2100 to 8100 tokens, 32 / 8 heads of 128, blocks of 16 (673 MB): 125 us,
// 5.4 TB/s, bound by reads with 8 waves a CU and 16 KB of each on their way (3 waves a
// SIMD, 44 registers spilled, 147 us).  Prompts of 600 to 1800 tokens over 2700 to 6800:
// 431 to 464 us, 650 TFLOP/s: 440 vector instructions beside 64 matrix instructions a
// tile of 64 tokens x 32 rows (128 of them widen codes, 32 are exponentials), the matrix
// cores busy a quarter of the time.  Prompts with nothing cached before them: one of 2048
// tokens 358 TFLOP/s, of 8192 506, 32 of 1024 329.  One request of 1030 tokens: 8 us and 4.5
// us for the merge, latency.
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

// Eight codes (two words) times a power of two as float16.
__device__ __forceinline__ half8 widen(uint32_t lo, uint32_t hi, float by = 1.0f) {
  half8 h;
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, by, false);
  const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, by, true);
  const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, by, false);
  const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, by, true);
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
  int64_t tiles;                         // most row tiles of a head
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

// Where a unit of a head's work lies.
struct Unit {
  int s;                                 // request
  int64_t first;                         // units before the request
  int tile0;                             // row tiles before the request
  Request r;
};

// The numbering of a head's work: sums over the requests by a lane each, or, from
// 65 requests on, over buckets of them by a thread each.
template <int M>
struct Plan {
  int64_t total, chunk;
  int tiles, per;                        // row tiles; requests a bucket
  int64_t upto;                          // up to 64 requests: units up to the lane's
  int tiles_upto;
  Request mine;
  const int64_t* before;                 // [257] units, and row tiles, before each bucket, in LDS
  const int* tiles_before;

  __device__ __forceinline__ void make(const AttendArgs& a, const Split& sp, int64_t* lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool few = a.S <= 64;
    per = few ? 1 : (a.S + 255) / 256;
    int64_t units = 0;
    int t = 0;
    mine = Request{0, 0, 0, 0, 0, 1};
    if (few) {
      if (lane < a.S) mine = request_of<M>(a, lane);
      units = (int64_t)mine.row_tiles * mine.kv_tiles;
      t = mine.row_tiles;
    } else {
      const int lo = tid * per, hi = lo + per < a.S ? lo + per : a.S;
      for (int s = lo; s < hi; ++s) {
        const Request r = request_of<M>(a, s);
        units += (int64_t)r.row_tiles * r.kv_tiles;
        t += r.row_tiles;
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int64_t y = __shfl_up(units, o);
      const int z = __shfl_up(t, o);
      if (lane >= o) {
        units += y;
        t += z;
      }
    }
    if (few) {
      upto = units;
      tiles_upto = t;
      total = __shfl(units, 63);
      tiles = __shfl(t, 63);
    } else {
      int* lds_t = (int*)(lds + 261);
      if (lane == 63) {
        lds[257 + wave] = units;
        lds_t[257 + wave] = t;
      }
      __syncthreads();
      for (int w = 0; w < wave; ++w) {
        units += lds[257 + w];
        t += lds_t[257 + w];
      }
      lds[tid + 1] = units;
      lds_t[tid + 1] = t;
      if (tid == 0) {
        lds[0] = 0;
        lds_t[0] = 0;
      }
      __syncthreads();
      before = lds;
      tiles_before = lds_t;
      total = lds[256];
      tiles = lds_t[256];
    }
    total = uniform(total);
    tiles = __builtin_amdgcn_readfirstlane(tiles);
    if (total < (int64_t(1) << 31))
      chunk = ((uint32_t)total + (uint32_t)sp.workers - 1) / (uint32_t)sp.workers;
    else chunk = (total + sp.workers - 1) / sp.workers;
    if (chunk < sp.least) chunk = sp.least;
  }

  static __device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
  }
  // The request of this lane's number, for all lanes.
  __device__ __forceinline__ void get(const AttendArgs& a, int s, Unit* u) const {
    u->s = s;
    if (a.S > 64) {
      u->r = request_of<M>(a, s);
      return;
    }
    const auto at = [&](int x) { return __builtin_amdgcn_readlane(x, s); };
    u->r = Request{at(mine.q0), at(mine.n), at(mine.len), at(mine.rows), at(mine.row_tiles),
                   at(mine.kv_tiles)};
  }
  // The request that holds unit x < total.
  __device__ __forceinline__ void find(const AttendArgs& a, int64_t x, Unit* u) const {
    if (a.S <= 64) {
      const int s = __builtin_ctzll(__ballot(upto > x));
      get(a, s, u);
      u->first = uniform(__shfl(upto, s)) - (int64_t)u->r.row_tiles * u->r.kv_tiles;
      u->tile0 = __builtin_amdgcn_readlane(tiles_upto, s) - u->r.row_tiles;
      return;
    }
    int b = 0;
#pragma unroll
    for (int step = 128; step > 0; step /= 2)
      if (before[b + step] <= x) b += step;
    u->first = before[b];
    u->tile0 = tiles_before[b];
    for (int s = b * per;; ++s) {
      get(a, s, u);
      const int64_t units = (int64_t)u->r.row_tiles * u->r.kv_tiles;
      if (x < u->first + units || s + 1 >= a.S) return;
      u->first += units;
      u->tile0 += u->r.row_tiles;
    }
  }
};

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

// The workspace: [head][worker][2] row tiles of M rows of sums, a worker's first and
// a later one that it does not end; for every row tile that lies in several ranges
// where its parts are, and how many row tiles there are.
struct Piece {
  int q0, row0, rows, at, n, pad;        // at: first worker * 2 + slot; the others' are slot 0
};
struct Partial {
  float* o;                              // [M][D]
  float2* ml;                            // [M]: m, l
};
template <int M, int D>
struct Space {
  char* ws;
  int64_t parts, tiles;                  // parts of all heads; most row tiles of a head
  __device__ __host__ Space(char* w, int64_t kv_heads, const Split& sp)
      : ws(w), parts(kv_heads * sp.workers * 2), tiles(sp.tiles) {}
  __device__ Partial part(const Split& sp, int head, int64_t i) const {
    i += (int64_t)head * sp.workers * 2;
    return {(float*)ws + i * M * D, (float2*)((float*)ws + parts * M * D) + i * M};
  }
  __device__ int* count() const { return (int*)(ws + parts * M * (D + 2) * 4); }
  __device__ Piece* piece(int head, int64_t tile) const {
    return (Piece*)(count() + 4) + head * tiles + tile;
  }
  int64_t bytes(int64_t kv_heads) const {
    return parts * M * (D + 2) * 4 + 16 + kv_heads * tiles * (int64_t)sizeof(Piece);
  }
};

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
  // Weights use float16 up to its end: a row's reference m lies 2^kBelow below the largest
  // when it moves, and moves where a weight would pass 2^kTop (with what is rounded,
  // 2^15.7 at most).  Float16 keeps 11 bits down to 2^-14, so of 16-bit types' weights those
  // above 2^-25 of the row's largest, and is off by 2^-25 below, 2^-36 of the largest.
  // A kBelow of 15 moves every row whose largest grows: prompts 431 us with 7, 433 with
  // 11, 438 with 13, 455 with 15 (3 of up to 2048 over 8192, 32 / 8 heads of 128).
  // Float32 does, and its low part is kept times kLow, against values over kLow, so that it
  // is never short of digits before the high one: 22 bits down to 2^-29, off by 2^-51 below.
  static constexpr float kTop = 15.25f, kBelow = kTwo ? 15.0f : 11.0f;
  static constexpr float kLow = 0x1p11f;

  half8 q[kParts][MT][NC];
  float factor[MT];                      // scale log2(e) 2^-k of the lane's query row, or < 0
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
      // a row that is not finite: equal scores, and NaN at the end where it has any
      factor[mt] = broken ? -1.0f : ldexpf(a.scale * kLog2e, -k);
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

  // What a tile of 64 tokens brings: the blocks of the lane's own tokens and of the key
  // row that it loads, 16-byte pieces of keys and values, the scales.
  struct Blocks {
    int own, key;
  };
  u32x4 kr[4][NI], vr[ND];
  float ks, vs;

  struct Cursor {
    const AttendArgs& a;
    const int32_t* table;
    const uint8_t *kb, *vb;
    int head, len, lane, shift;
    __device__ __forceinline__ Cursor(const AttendArgs& a_, int s, int len_, int head_, int lane_)
        : a(a_), table(a_.table + (int64_t)s * a_.table_ld), head(head_), len(len_), lane(lane_),
          shift(__builtin_ctz(a_.block_size)) {
      kb = a.k.codes + (int64_t)head * a.block_size * D + (lane >> 4) * 16;
      vb = a.v.codes + ((int64_t)head * D + (lane & 15)) * a.block_size;
    }
    __device__ __forceinline__ int own(int kt) const { return kt * kTile + (lane >> 4) * 16; }
    __device__ __forceinline__ int key(int kt) const { return kt * kTile + (lane & 15) / 4 * 16; }
    __device__ __forceinline__ Blocks blocks(int kt) const {
      Blocks b{-1, -1};
      if (own(kt) < len) b.own = table[own(kt) >> shift];
      if (key(kt) < len) b.key = table[key(kt) >> shift];
      return b;
    }
    __device__ __forceinline__ bool there(int block) const {
      return (unsigned)block < (unsigned)a.num_blocks;
    }
  };
  // Mostly one row tile a request: nothing reads its blocks again, and they need not stay
  // in the caches (64 requests of up to 8192: 126 us, through them 133).
  static __device__ __forceinline__ u32x4 load16(const uint8_t* p) {
    if constexpr (MT == 1) return __builtin_nontemporal_load((const u32x4*)p);
    return *(const u32x4*)p;
  }
  __device__ __forceinline__ void load_keys(const Cursor& c, const Blocks& b, int kt) {
    const int key = c.there(b.key) ? b.key : 0, own = c.there(b.own) ? b.own : 0;
    const int o = (c.key(kt) & (c.a.block_size - 1)) + (c.lane & 3);
    const uint8_t* p = c.kb + (int64_t)key * c.a.k.stride + o * D;
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
      for (int i = 0; i < NI; ++i) kr[tt][i] = load16(p + tt * 4 * D + i * 64);
    ks = c.a.k.scale[(int64_t)own * c.a.kv_heads + c.head];
    vs = c.a.v.scale[(int64_t)own * c.a.kv_heads + c.head];
  }
  __device__ __forceinline__ void load_values(const Cursor& c, const Blocks& b, int kt) {
    const int own = c.there(b.own) ? b.own : 0;
    const uint8_t* p =
        c.vb + (int64_t)own * c.a.v.stride + (c.own(kt) & (c.a.block_size - 1));
#pragma unroll
    for (int d = 0; d < ND; ++d) vr[d] = load16(p + d * 16 * c.a.block_size);
  }

  // Tiles kt0 .. kt1 - 1.  `now` and `next`: the blocks of kt0, whose keys and values
  // are on their way, and of kt0 + 1.  The next tile's keys are asked for when this
  // one's are used up, its values behind this one's, its blocks a tile before.
  __device__ __forceinline__ void run(const Cursor& cur, Blocks now, Blocks next, int kt0, int kt1,
                                      int open) {
    const int j = cur.lane >> 4;
    for (int kt = kt0; kt < kt1; ++kt) {
      const int base = kt * kTile, tj = base + j * 16;
      const bool there = cur.there(now.own);
      Blocks after{-1, -1};
      if (kt + 2 < kt1) after = cur.blocks(kt + 2);
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
      ks = clamp_scale(ks);
      vs = clamp_scale(vs);
      const bool no_keys = there && ks != ks, no_values = there && vs != vs;
      const float kf = ks != ks ? 1.0f : ks;
      const float vf = vs != vs ? 1.0f : vs;
      const float lv = __builtin_amdgcn_logf(vf), iv = __builtin_amdgcn_rcpf(vf);
      __builtin_amdgcn_sched_barrier(0);
      if (kt + 1 < kt1) load_keys(cur, next, kt + 1);
      __builtin_amdgcn_sched_barrier(0);
      // tokens behind a row's own, behind the length, or in no block
      const bool all = __all(there) && base + kTile <= open;
      if (!all) {
        const int valid = there ? cur.len - tj : 0;
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
        float cf = factor[mt] * kf;
        if (cf < 0x1p-126f) cf = 0x1p-126f;          // -inf * 0 would be NaN; a broken row
        want[mt] = row_max4(fmaf(top, cf, lv));
        moves |= want[mt] - m[mt] > kTop;
      }
      if (__any(moves)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // (far from 0 the difference may be rounded to more)
          float low = want[mt] - kBelow;
          if (!(want[mt] - low <= kTop)) low = want[mt];
          const float now = fmaxf(m[mt], low);
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
        float cf = factor[mt] * kf;
        if (cf < 0x1p-126f) cf = 0x1p-126f;
        float shiftv = lv - (m[mt] == kNegInf ? 0.0f : m[mt]);
        // The product below is exact and m is rounded: they are apart by up to 2^-24 |m|.
        // Where that is much (a quarter: weights stay below 2^16) the scores are rounded first,
        // as m was.
        if (__any(fabsf(m[mt]) > 0x1p22f && m[mt] != kNegInf)) {
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
              p[kParts - 1][mt][tt >> 1][(tt & 1) * 4 + e] = (_Float16)((w - (float)(_Float16)w) * kLow);
          }
        }
        l[mt] = fmaf(sum, iv, l[mt]);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const half8 v8 =
                widen(vr[d][half * 2], vr[d][half * 2 + 1], part == 0 ? 1.0f : 1.0f / kLow);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][d] = mma(v8, p[part][mt][half], o[mt][d]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (kt + 1 < kt1) load_values(cur, next, kt + 1);
      __builtin_amdgcn_sched_barrier(0);
      now = next;
      next = after;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] = row_sum4(l[mt]);
      if (factor[mt] < 0.0f && l[mt] != 0.0f) l[mt] = __builtin_nanf("");
    }
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
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attend_kernel(AttendArgs a, Split sp, char* ws) {
  constexpr int M = 16 * MT;
  __shared__ int64_t lds[261 + 131];
  const int head = blockIdx.x % a.kv_heads, lane = threadIdx.x & 63;
  clear_outside<T>(a, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
  if (a.S == 0) return;
  Plan<M> plan;
  plan.make(a, sp, lds);
  const Space<M, D> space(ws, a.kv_heads, sp);
  if (blockIdx.x == 0 && threadIdx.x == 0) *space.count() = plan.tiles;
  const int64_t worker = (int64_t)(blockIdx.x / a.kv_heads) * 4 +
                         __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int64_t u = worker * plan.chunk;
  const int64_t u0 = u, u1 = u + plan.chunk < plan.total ? u + plan.chunk : plan.total;
  if (u >= u1) return;
  const int group = a.q_heads / a.kv_heads;
  Unit at;
  plan.find(a, u, &at);
  while (u < u1) {
    const Request& r = at.r;
    const int64_t units = (int64_t)r.row_tiles * r.kv_tiles;
    if (u >= at.first + units) {
      at.first += units;
      at.tile0 += r.row_tiles;
      if (at.s + 1 >= a.S) return;
      plan.get(a, at.s + 1, &at);
      continue;
    }
    const int64_t in = u - at.first;
    const int t = in < (int64_t(1) << 31) ? (int)((uint32_t)in / (uint32_t)r.kv_tiles)
                                          : (int)(in / r.kv_tiles);
    const int64_t first = at.first + (int64_t)t * r.kv_tiles;
    const int need = tiles_of<M>(r, t, group);
    const int64_t end = first + r.kv_tiles < u1 ? first + r.kv_tiles : u1;
    const int kt0 = (int)(u - first), kt1 = (int)(end - first < need ? end - first : need);
    if (kt0 < kt1) {
      typedef RowTile<T, D, MT> Tile;
      Tile tile;
      const typename Tile::Cursor cur(a, at.s, r.len, head, lane);
      typename Tile::Blocks now{-1, -1}, next{-1, -1};
      if (r.len > 0) {
        now = cur.blocks(kt0);
        if (kt0 + 1 < kt1) next = cur.blocks(kt0 + 1);
        tile.load_keys(cur, now, kt0);
        tile.load_values(cur, now, kt0);
      }
      tile.load_queries(a, r, t, head, lane);
      if (r.len > 0) tile.run(cur, now, next, kt0, kt1, seen_of(r, t * M, group));
      if (kt0 == 0 && kt1 == need) tile.finish(a, r, t, head, lane);
      else tile.save(space.part(sp, head, worker * 2 + (u > u0)), r, t, lane);
      if (kt0 == 0 && lane == 0) {
        const int64_t last = first + need - 1;
        const int n = kt1 == need ? 0
                                  : (int)((last < (int64_t(1) << 31) && plan.chunk < (int64_t(1) << 31)
                                               ? (uint32_t)last / (uint32_t)plan.chunk
                                               : last / plan.chunk) -
                                          worker);
        const int rows = r.rows - t * M < M ? r.rows - t * M : M;
        // more row tiles than there is room for have offsets that decrease
        if (at.tile0 + t < sp.tiles)
          *space.piece(head, at.tile0 + t) =
            Piece{r.q0, t * M, rows, (int)(worker * 2 + (u > u0)), n, 0};
      }
    }
    u = end;
  }
}

// Merges the parts of a row tile that lies in several ranges.  Workgroup (t, head, y):
// rows R y .. of row tile t, R of them a time; what threads are left share the parts.
constexpr int kMergeRows = 1024;         // floats of a row times rows a workgroup
template <typename T, int D, int MT, int NT>
__global__ __launch_bounds__(NT) void merge_kernel(AttendArgs a, Split sp, char* ws) {
  constexpr int M = 16 * MT, L = D / 4, R = kMergeRows / D, G0 = NT / (R * L);
  __shared__ f32x4 sums[NT];
  __shared__ float2 mls[NT / L];
  const Space<M, D> space(ws, a.kv_heads, sp);
  const int head = blockIdx.y, i0 = blockIdx.z * R, group = a.q_heads / a.kv_heads;
  const int all = *space.count();
  for (int64_t tile = blockIdx.x; tile < sp.tiles; tile += gridDim.x) {
    // (read before it is known whether there is one: its place is there)
    const Piece x = *space.piece(head, tile);
    if (tile >= all || x.n == 0 || i0 >= x.rows) continue;
    const int here = x.rows - i0 < R ? x.rows - i0 : R;
    // fewer rows: more groups, each with every G-th part
    int G = G0, span = R;
    while (span / 2 >= here) {
      span /= 2;
      G *= 2;
    }
    const int lanes = threadIdx.x / L, i = i0 + lanes % span, g = lanes / span;
    const int d = threadIdx.x % L * 4;
    float m = kNegInf, l = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    if (i < x.rows) {
      const int first = x.at / 2;
      // a part's place: its worker's slot 0, but for the first
      const auto part = [&](int k) {
        return space.part(sp, head, k == 0 ? x.at : (first + k) * 2);
      };
#pragma unroll 4
      for (int k = g; k <= x.n; k += G) {
        const Partial p = part(k);
        const float2 ml = p.ml[i];
        const f32x4 v = *(const f32x4*)(p.o + i * D + d);
        const float top = fmaxf(m, ml.x), ref = top == kNegInf ? 0.0f : top;
        const float keep = exp2_fast(m - ref), f = exp2_fast(ml.x - ref);
        l = fmaf(ml.y, f, l * keep);
        o = o * keep + v * f;
        m = top;
      }
    }
    if (G > 1) {
      __syncthreads();                   // the sums of the tile before are used
      sums[threadIdx.x] = o;
      if (d == 0) mls[lanes] = make_float2(m, l);
      __syncthreads();
      if (g == 0) {
        float top = m;
        for (int k = 1; k < G; ++k) top = fmaxf(top, mls[lanes + k * span].x);
        const float ref = top == kNegInf ? 0.0f : top, f0 = exp2_fast(m - ref);
        o = o * f0;
        l *= f0;
        for (int k = 1; k < G; ++k) {
          const float2 ml = mls[lanes + k * span];
          const float f = exp2_fast(ml.x - ref);
          l = fmaf(ml.y, f, l);
          o += sums[threadIdx.x + k * span * L] * f;
        }
        m = top;
      }
    }
    if (g > 0 || i >= x.rows) continue;
    const int row = x.row0 + i, token = row / group;
    const int h = head * group + row - token * group;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    store4((T*)a.out + (int64_t)(x.q0 + token) * a.out_ld + (int64_t)h * D + d, o[0] * inv,
           o[1] * inv, o[2] * inv, o[3] * inv);
    if (a.lse && d == 0)
      a.lse[(int64_t)(x.q0 + token) * a.q_heads + h] =
          l == 0.0f ? kNegInf : (float)(kLn2 * ((double)m + log2((double)l)));
  }
}

// Row tiles of 16 or 32 rows, by the mean rows of a request: 32 share what a tile of
// tokens costs (3 prompts of up to 2048 over 8192, 32 / 8 heads of 128 bf16: 439 us, by
// 16 1308).  Float32 of dim 128 and 256 spills registers with 32, and takes them from
// three 16s on only (16 x 5 over 8192, 32 / 8 heads of 128: by 16 75 us, by 32 92; 7 x
// 3 over 4000, 8 / 1 of 256: 26 and 33; 3 prompts of up to 1024, 8 / 2 of 256: 400 and 320,
// all with float32's low weights at the high ones' scale; the last is 291 now).
int row_tiles_of(int64_t T, int64_t S, int64_t group, int64_t dim, lik_dtype dtype) {
  const int64_t most = dtype == LIK_F32 && dim > 64 ? 32 : 16;
  return S > 0 && T * group <= most * S ? 1 : 2;
}
Split split_of(int64_t T, int64_t S, int64_t q_heads, int64_t kv_heads, int64_t dim,
               lik_dtype dtype) {
  // Eight a CU, as many as are resident at dims 64 and 128.  At 256 four are, and the others
  // follow them: fewer would halve the workspace and the merge there (not tried).
  constexpr int kWaves = 2048;
  const int64_t group = q_heads / kv_heads, M = 16 * row_tiles_of(T, S, group, dim, dtype);
  const int64_t w = (kWaves / 4 + kv_heads - 1) / kv_heads * 4;
  // every request has a row tile that is not full at most
  const int64_t tiles = T * group / M + (S < T ? S : T);
  return {(int)w, 1, tiles};
}

template <typename T, int D, int MT>
hipError_t attend_t(const AttendArgs& a, char* ws, hipStream_t s) {
  const Split sp = split_of(a.T, a.S, a.q_heads, a.kv_heads, a.dim, a.dtype);
  hipLaunchKernelGGL((attend_kernel<T, D, MT>), dim3(sp.workers / 4 * a.kv_heads), dim3(256), 0, s,
                     a, sp, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 0) return e;
  // few row tiles leave room for more threads on each
  const dim3 grid((unsigned)(sp.tiles < 65536 ? sp.tiles : 65536), a.kv_heads,
                  16 * MT * D / kMergeRows);
  if (sp.tiles * a.kv_heads <= 512)
    hipLaunchKernelGGL((merge_kernel<T, D, MT, 1024>), grid, dim3(1024), 0, s, a, sp, ws);
  else
    hipLaunchKernelGGL((merge_kernel<T, D, MT, 256>), grid, dim3(256), 0, s, a, sp, ws);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t attend_d(const AttendArgs& a, char* ws, hipStream_t s) {
  if (row_tiles_of(a.T, a.S, a.q_heads / a.kv_heads, a.dim, a.dtype) == 1)
    return attend_t<T, D, 1>(a, ws, s);
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
  const Split sp = split_of(T, S, q_heads, kv_heads, dim, dtype);
  const bool one = row_tiles_of(T, S, q_heads / kv_heads, dim, dtype) == 1;
  const auto bytes = [&](auto d) -> int64_t {
    constexpr int D = decltype(d)::value;
    return one ? Space<16, D>(nullptr, kv_heads, sp).bytes(kv_heads)
               : Space<32, D>(nullptr, kv_heads, sp).bytes(kv_heads);
  };
  if (dim == 64) return (size_t)bytes(std::integral_constant<int, 64>());
  if (dim == 128) return (size_t)bytes(std::integral_constant<int, 128>());
  return (size_t)bytes(std::integral_constant<int, 256>());
}

hipError_t run_attend(const AttendArgs& a, char* ws, hipStream_t s) {
  if (a.dtype == LIK_F16) return attend_type<_Float16>(a, ws, s);
  if (a.dtype == LIK_BF16) return attend_type<__bf16>(a, ws, s);
  return attend_type<float>(a, ws, s);
}

}  // namespace lik

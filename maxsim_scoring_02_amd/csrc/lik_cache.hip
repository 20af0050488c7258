// Block tables and writes of the 8-bit cache (include/lik_cache.h).
#include <hip/hip_runtime.h>

#include <type_traits>

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

// Sums of blocks and tokens are unsigned and stay at the largest number: what a pool or
// a slot map can hold is far below, and beyond it nothing is granted or stored.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
  return __builtin_elementwise_add_sat(a, b);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
  return add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false));
}
// Sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = dpp_add<0x111, 0xf>(v);            // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);            // the last of a row to the next
  return dpp_add<0x143, 0xc>(v);         // of the lower half to the upper
}

// Three running sums over a workgroup: before this thread, and of all.  Two places in
// LDS in turn: one meeting a call.
struct Sums {
  uint32_t x, y, z;
};
typedef Sums ScanLds[2][kTablesThreads / 64];
__device__ __forceinline__ Sums scan3(Sums v, ScanLds& lds, int& turn, Sums* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Sums upto{wave_scan(v.x), wave_scan(v.y), wave_scan(v.z)};
  turn ^= 1;
  if (lane == 63) lds[turn][wave] = upto;
  __syncthreads();
  Sums r{0, 0, 0}, sum{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kTablesThreads / 64; ++w) {
    if (w == wave) r = sum;
    const Sums o = lds[turn][w];
    sum = Sums{add(sum.x, o.x), add(sum.y, o.y), add(sum.z, o.z)};
  }
  *all = sum;
  // the lanes before this one
  const int before = lane == 0 ? 64 : lane - 1;
  const uint32_t x = __shfl(upto.x, before), y = __shfl(upto.y, before), z = __shfl(upto.z, before);
  if (lane == 0) return r;
  return Sums{add(r.x, x), add(r.y, y), add(r.z, z)};
}

// The last entry of a rising array that is at most x; the first is.
__device__ __forceinline__ int last_at_most(const uint32_t* v, uint32_t x) {
  int b = 0;
#pragma unroll
  for (int step = kTablesThreads / 2; step > 0; step /= 2)
    if (v[b + step] <= x) b += step;
  return b;
}
// A place in the ring; a consistent pool goes round its end once at most.
__device__ __forceinline__ int ring_at(uint32_t i, int N) {
  if (i >= (uint32_t)N) i -= N;
  return (int)(i < (uint32_t)N ? i : i % N);
}

// One launch.  Workgroup (x, y) takes the requests 256 x .. 256 x + 255 (and further
// ones, gridDim.x * 256 apart), and of their table entries and slots every
// gridDim.y-th 256: it sums what all requests before ask for by itself, which is a
// few loads a thread for as many requests as a batch has, and needs no workgroup to
// wait for another.  The workgroup that is last to have read the pool's state
// (counted in ring_state[2], which it sets back) moves it.  Blocks to take and room
// for blocks given back lie apart in the ring, so entries are independent.
// 64 requests that take 5 tokens each 6 us, 100000 slots of 12 that come back 7 us:
// latency, three meetings of the workgroup.  1000 prompts, a million slots (4 MB) in 17
// us, their blocks back in 9 us.
__global__ __launch_bounds__(kTablesThreads) void tables_kernel(TablesArgs a) {
  __shared__ ScanLds lds;
  __shared__ uint32_t entry0[kTablesThreads], token0[kTablesThreads];
  __shared__ int s_old[kTablesThreads], s_have[kTablesThreads], s_need[kTablesThreads];
  __shared__ uint32_t s_ring[kTablesThreads];    // where its blocks come from or go to
  __shared__ int is_last, s_state[2];
  constexpr uint32_t kNotGranted = ~0u;
  const int tid = threadIdx.x, bs = a.block_size, N = a.num_blocks;
  const int shift = __builtin_ctz(bs);
  int turn = 0;
  // one thread reads the state, and counts once it has it
  if (tid == 0) {
    const int h = a.state[0], f = a.state[1], n = (int)(gridDim.x * gridDim.y);
    s_state[0] = N > 0 && h > 0 ? h % N : 0;
    s_state[1] = f < 0 ? 0 : (f > N ? N : f);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    is_last = n == 1 || atomicAdd(&a.state[2], 1) == n - 1;
  }
  const auto change = [&](int s) {
    Change c{0, 0, 0, 0, false};
    if (s < a.S) c = change_of(a, s, shift);
    return c;
  };
  const auto granted = [&](const Change& c, uint32_t before) {
    const uint32_t ask = c.ask();
    return c.fits && (ask == 0 || add(before, ask) <= (uint32_t)s_state[1]);
  };

  Sums upto{0, 0, 0};                            // asked, given, grown before s0
  uint32_t taken = 0, back = 0;                  // of all, where one workgroup sees all
  int done = 0;
  for (int s0 = blockIdx.x * kTablesThreads; s0 < a.S; s0 += gridDim.x * kTablesThreads) {
    Sums all;
    Change c = change(s0 + tid);
    if (s0 > done) {                             // sums of the requests between
      Sums mine{0, 0, 0};
      for (int s = done + tid; s < s0; s += kTablesThreads) {
        const Change o = change_of(a, s, shift);
        mine = Sums{add(mine.x, o.ask()), add(mine.y, o.give()), add(mine.z, o.grown())};
      }
      scan3(mine, lds, turn, &all);
      upto = Sums{add(upto.x, all.x), add(upto.y, all.y), add(upto.z, all.z)};
    }
    const int s = s0 + tid;
    const Sums before = scan3(Sums{(uint32_t)c.ask(), (uint32_t)c.give(), (uint32_t)c.grown()}, lds,
                              turn, &all);       // s_state is there too now
    const int head = s_state[0], free_blocks = s_state[1];
    const uint32_t start = add(upto.x, before.x), rel = add(upto.y, before.y);
    const bool ok = granted(c, start);
    const uint32_t ask = ok ? c.ask() : 0, give = ok ? c.give() : 0;
    Sums moved;
    const Sums entry = scan3(Sums{ask + give, ask, give}, lds, turn, &moved);
    taken = add(taken, moved.y);
    back = add(back, moved.z);
    entry0[tid] = entry.x;
    token0[tid] = before.z;
    s_old[tid] = c.old_len;
    s_have[tid] = c.have;
    s_need[tid] = c.need;
    s_ring[tid] = !ok ? kNotGranted : (ask ? head + start : add(head + free_blocks, rel));
    if (s < a.S && blockIdx.y == 0) {
      const uint32_t first = add(upto.z, before.z);
      a.granted[s] = ok ? c.new_len : c.old_len;
      a.offsets[s] = first < INT32_MAX ? (int)first : INT32_MAX;
    }
    __syncthreads();
    // table entries (their number may be next to 2^32, where a step further is not)
    for (uint64_t at = blockIdx.y * kTablesThreads + tid; at < moved.x;
         at += gridDim.y * kTablesThreads) {
      const uint32_t e = (uint32_t)at;
      const int i = last_at_most(entry0, e), k = (int)(e - entry0[i]);
      int32_t* row = a.table + (s0 + i) * a.table_ld;
      if (s_need[i] > s_have[i]) {
        row[s_have[i] + k] = a.ring[ring_at(s_ring[i] + k, N)];
      } else {
        if (N > 0) a.ring[ring_at(s_ring[i] + k, N)] = row[s_need[i] + k];
        row[s_need[i] + k] = -1;
      }
    }
    // slots, four neighbours a thread
    const uint32_t most = upto.z < (uint32_t)a.T ? a.T - upto.z : 0;
    const uint32_t here = all.z < most ? all.z : most;
    for (uint32_t e = (blockIdx.y * kTablesThreads + tid) * 4; e < here;
         e += gridDim.y * kTablesThreads * 4) {
      typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));
      i32x4 slot;
      int i = last_at_most(token0, e), from = -1, which = -1, b = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        while (i + 1 < kTablesThreads && token0[i + 1] <= e + j) ++i;
        const int p = s_old[i] + (int)(e + j - token0[i]), at = p >> shift;
        if (from != i || which != at) {          // another block than the last
          from = i;
          which = at;
          b = -1;
          if (e + j < here && s_ring[i] != kNotGranted)
            b = at < s_have[i] ? a.table[(s0 + i) * a.table_ld + at]
                               : a.ring[ring_at(s_ring[i] + at - s_have[i], N)];
        }
        slot[j] = (unsigned)b < (unsigned)N ? (b << shift) + (p & (bs - 1)) : -1;
      }
      int32_t* out = a.slots + upto.z + e;
      if (e + 3 < here) *(i32x4*)out = slot;
      else
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < here) out[j] = slot[j];
    }
    upto = Sums{add(upto.x, all.x), add(upto.y, all.y), add(upto.z, all.z)};
    done = s0 + kTablesThreads;
    if (done + (int)(gridDim.x - 1) * kTablesThreads < a.S) __syncthreads();   // the arrays again
  }
  __syncthreads();
  // tokens of the requests behind, then what no request has
  uint32_t tokens = upto.z;
  if (done < a.S) {
    Sums mine{0, 0, 0}, all;
    for (int s = done + tid; s < a.S; s += kTablesThreads)
      mine.x = add(mine.x, change_of(a, s, shift).grown());
    scan3(mine, lds, turn, &all);
    tokens = add(tokens, all.x);
  }
  const int64_t linear = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t threads = (int64_t)gridDim.x * gridDim.y * kTablesThreads;
  for (int64_t i = tokens + linear * kTablesThreads + tid; i < a.T; i += threads) a.slots[i] = -1;
  if (linear == 0 && tid == 0) a.offsets[a.S] = tokens < INT32_MAX ? (int)tokens : INT32_MAX;
  if (!is_last) return;
  if (gridDim.x > 1) {                           // what all took and gave back
    Sums all, x;
    uint32_t asked = 0;
    taken = back = 0;
    for (int s0 = 0; s0 < a.S; s0 += kTablesThreads) {
      const Change c = change(s0 + tid);
      const Sums before = scan3(Sums{(uint32_t)c.ask(), 0, 0}, lds, turn, &all);
      const bool ok = granted(c, add(asked, before.x));
      scan3(Sums{0, ok ? (uint32_t)c.ask() : 0, ok ? (uint32_t)c.give() : 0}, lds, turn, &x);
      asked = add(asked, all.x);
      taken = add(taken, x.y);
      back = add(back, x.z);
    }
  }
  if (tid == 0) {
    if (N > 0) {
      const uint32_t now = add(s_state[1] - taken, back);
      a.state[0] = ring_at(s_state[0] + taken, N);
      a.state[1] = (int)(now > (uint32_t)N ? N : now);
    }
    a.state[2] = 0;
  }
}

// ---------------------------------------------------------------------------
// appends
// ---------------------------------------------------------------------------

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

// Four numbers of at most 448 as codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}
__device__ __forceinline__ uint32_t recode(uint32_t x, float k) {
  return to_codes(__builtin_amdgcn_cvt_f32_fp8((int)x, 0) * k, __builtin_amdgcn_cvt_f32_fp8((int)x, 1) * k,
                  __builtin_amdgcn_cvt_f32_fp8((int)x, 2) * k, __builtin_amdgcn_cvt_f32_fp8((int)x, 3) * k);
}
// An unsigned maximum of float32 magnitudes, or of two 16-bit ones in each word: what is
// not finite is larger than all that is.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
  return y > v ? y : v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max<0xB1>(v);                  // quad_perm 1,0,3,2
  v = dpp_max<0x4E>(v);                  // quad_perm 2,3,0,1
  v = dpp_max<0x141>(v);                 // row_half_mirror
  v = dpp_max<0x140>(v);                 // row_mirror
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = r[0] > r[1] ? r[0] : r[1];
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __builtin_amdgcn_readfirstlane((int)(r[0] > r[1] ? r[0] : r[1]));
}

// Four tokens of a row piece: 8 numbers of a lane each.
template <typename T>
struct Quad {
  static constexpr int W = sizeof(T) / 2;        // 16-byte pieces a token
  u32x4 raw[4][W];
  // Two numbers over a power of two, rounded to nearest even, into the lower or upper
  // half of a word of codes.
  template <bool Upper>
  static __device__ __forceinline__ s16x2 codes2(s16x2 old, uint32_t a, uint32_t b, float scale) {
    if constexpr (W == 2)
      return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(old, __uint_as_float(a), __uint_as_float(b),
                                                      scale, Upper);
    else if constexpr (__is_same(T, __bf16)) {
      typedef __bf16 pair __attribute__((ext_vector_type(2)));
      return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, __builtin_bit_cast(pair, a), scale, Upper);
    } else {
      typedef _Float16 pair __attribute__((ext_vector_type(2)));
      return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(old, __builtin_bit_cast(pair, a), scale, Upper);
    }
  }
  // Dims 4 i .. 4 i + 3 of token k.
  __device__ __forceinline__ uint32_t dims4(int k, int i, float scale) const {
    s16x2 r = {0, 0};
    if constexpr (W == 2) {
      r = codes2<false>(r, raw[k][i][0], raw[k][i][1], scale);
      r = codes2<true>(r, raw[k][i][2], raw[k][i][3], scale);
    } else {
      r = codes2<false>(r, raw[k][0][2 * i], 0, scale);
      r = codes2<true>(r, raw[k][0][2 * i + 1], 0, scale);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
  // Dim i of the four tokens.
  __device__ __forceinline__ uint32_t tokens4(int i, float scale) const {
    s16x2 r = {0, 0};
    if constexpr (W == 2) {
      r = codes2<false>(r, raw[0][i / 4][i % 4], raw[1][i / 4][i % 4], scale);
      r = codes2<true>(r, raw[2][i / 4][i % 4], raw[3][i / 4][i % 4], scale);
    } else {
      const uint32_t pick = i % 2 ? 0x07060302u : 0x05040100u;
      const auto both = [&](int k) {
        return __builtin_amdgcn_perm(raw[k + 1][0][i / 2], raw[k][0][i / 2], pick);
      };
      r = codes2<false>(r, both(0), 0, scale);
      r = codes2<true>(r, both(2), 0, scale);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
  // The largest magnitude's bits as float32's.
  __device__ __forceinline__ uint32_t largest() const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = raw[k][j][i];
          if constexpr (W == 2) {
            const uint32_t x = u & 0x7fffffffu;
            m = x > m ? x : m;
          } else {
            const u16x2 x = __builtin_bit_cast(u16x2, u & 0x7fff7fffu), y = __builtin_bit_cast(u16x2, m);
            m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
          }
        }
    if constexpr (W == 1) {
      const uint16_t hi = (uint16_t)(m >> 16), lo = (uint16_t)m, x = hi > lo ? hi : lo;
      if constexpr (__is_same(T, __bf16)) m = (uint32_t)x << 16;
      else m = __float_as_uint((float)__builtin_bit_cast(_Float16, x)) & 0x7fffffffu;
    }
    return m;
  }
};

// The tokens of a call that go to one block, first of them at t: a run.  A group of
// `waves` waves (1, 2 or 4) does a run for one head and one of keys and values, in
// tiles aligned to the block: a lane has 8 dims of 4 neighbouring tokens, so that four
// codes of a dim are one word of the value's block, and 8 of a token two words of the
// key's.  A tile of keys is as wide as a token, one of values as long as 64 tokens or
// the block, so that both are stored in whole lines.  The group takes the largest
// number, then the scale, then the codes; a wave with one tile keeps it in registers
// meanwhile, one with more reads them again from the cache.  A scale is a power of
// two, so one instruction scales, rounds and packs two codes.  18437 tokens of 8 heads of
// 128, f16, blocks of 64 (113 MB): 25 us, 4.5 TB/s, f32 (189 MB) 43 us, 4.4 TB/s; 64 single
// tokens 5.5 us, latency (one more where scales grow and blocks of 64 are coded again).
// log2 of the lanes side by side in a tile of values: as few as there are dims for, so
// that a tile is as long as 64 tokens or the block.
__device__ __forceinline__ int append_side(int dim, int shift) {
  const int most = dim == 64 ? 3 : 4, least = 8 - (shift < 6 ? shift : 6);
  return least < most ? least : most;
}

template <typename T, int D>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, int waves, int tokens) {
  __shared__ uint32_t s_max[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int bs = a.block_size, shift = __builtin_ctz(bs);
  const auto block_of = [&](int slot) {
    return slot < 0 || (slot >> shift) >= a.num_blocks ? -1 : slot >> shift;
  };
  const int per = 4 / waves, items = a.heads * 2;
  for (int64_t at0 = (int64_t)blockIdx.y * tokens; at0 < a.T; at0 += (int64_t)gridDim.y * tokens) {
    const int t0 = (int)at0;
    // the slots from the workgroup's first on, and which of its tokens begin a run
    const int mine = t0 + lane < a.T ? a.slots[t0 + lane] : -1;
    int prior = __shfl_up(mine, 1);        // by all lanes: one that is not there gives nothing
    if (lane == 0 && t0 > 0) prior = a.slots[t0 - 1];
    const int my_block = block_of(mine);
    uint64_t begins = __ballot(lane < tokens && my_block >= 0 &&
                               (t0 + lane == 0 || my_block != block_of(prior)));
    for (; begins; begins &= begins - 1) {
      const int i0 = __builtin_ctzll(begins), t = t0 + i0;
      const int slot0 = __builtin_amdgcn_readlane(mine, i0), b = block_of(slot0);
      // the run: how long, and whether slots follow each other
      uint64_t out = ~__ballot(my_block == b) >> i0;
      int n = out ? __builtin_ctzll(out) : 64;
      if (n > 64 - i0) n = 64 - i0;
      const bool in = lane >= i0 && lane < i0 + n;
      bool follows = __all(!in || mine == slot0 + lane - i0);
      bool zero = __any(in && (mine & (bs - 1)) == 0);     // the block's first slot is written
      for (int more = i0 + n == 64 ? 64 : 0; more == 64; n += more) {
        const int i = t + n + lane, slot = i < a.T ? a.slots[i] : -1;
        out = ~__ballot(block_of(slot) == b);
        more = out ? __builtin_ctzll(out) : 64;
        follows &= __all(lane >= more || slot == slot0 + n + lane);
        zero |= __any(lane < more && (slot & (bs - 1)) == 0);
      }
      const int o0 = slot0 & (bs - 1);
      for (int item0 = blockIdx.x * per; item0 < items; item0 += gridDim.x * per) {
        // the same number of rounds for every wave: they meet below
        const int item = item0 + wave / waves;
        const bool works = item < items;
        const int h = works ? item >> 1 : 0, part = item & 1, w = wave & (waves - 1);
        const CachePart c = a.part[part];
        const T* x = (const T*)a.x[part] + (int64_t)h * D;
        uint8_t* codes = c.codes + (int64_t)b * c.stride + (int64_t)h * bs * D;
        float* scale = c.scale + (int64_t)b * a.heads + h;
        const int64_t ld = a.ld[part];
        // lanes of a tile side by side in dims, 8 each; tokens and dims of the lane
        const int side = part ? append_side(D, shift) : __builtin_ctz(D / 8);   // log2
        const int wide = __builtin_ctz(D / 8) - side, length = 8 - side;        // dims, tokens
        const int q = (lane >> side) * 4, d0 = (lane & ((1 << side) - 1)) * 8;
        const int first = o0 >> length;
        const int end = works && follows ? (((o0 + n - 1) >> length) + 1 - first) << wide : 0;
        Quad<T> v;
        const auto token_of = [&](int tile) { return ((first + (tile >> wide)) << length) + q; };
        const auto dim_of = [&](int tile) { return d0 + ((tile & ((1 << wide) - 1)) << (side + 3)); };
        // whether all of a tile's tokens are the run's
        const auto inside = [&](int tile) {
          const int o = (first + (tile >> wide)) << length;
          return o >= o0 && o + (1 << length) <= o0 + n;
        };
        const auto load = [&](int tile) {
          const int i = token_of(tile) - o0;
          const T* p = x + (t + i) * ld + dim_of(tile);
          if (inside(tile)) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int j = 0; j < Quad<T>::W; ++j) v.raw[k][j] = *((const u32x4*)(p + k * ld) + j);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int j = 0; j < Quad<T>::W; ++j) {
                v.raw[k][j] = u32x4{0, 0, 0, 0};
                if (i + k >= 0 && i + k < n) v.raw[k][j] = *((const u32x4*)(p + k * ld) + j);
              }
          }
        };
        uint32_t top = 0;
        const float was = works ? *scale : 1.0f;
        int here = w - waves;              // the tile in registers; none yet
        for (int tile = w; tile < end; tile += waves) {
          load(here = tile);
          const uint32_t m = v.largest();
          top = m > top ? m : top;
        }
        if (works && !follows)             // tokens in any order
          for (int i = w * 64 + lane; i < n * D; i += waves * 64) {
            const float f = (float)x[(int64_t)(t + i / D) * a.ld[part] + i % D];
            const uint32_t m = __float_as_uint(f) & 0x7fffffffu;
            top = m > top ? m : top;
          }
        top = wave_max_u32(top);
        if (waves > 1) {
          if (lane == 0) s_max[wave] = top;
          __syncthreads();
          for (int i = wave & ~(waves - 1), end = i + waves; i < end; ++i)
            top = s_max[i] > top ? s_max[i] : top;
        }
        const bool bad = top >= 0x7f800000u;
        float now = scale_of(bad ? 0.0f : __uint_as_float(top));
        if (!zero) now = grown_scale(was, now);
        if (bad) now = __builtin_nanf("");
        const bool none = now != now;      // all codes are 0 then
        // in any order, or beyond the largest scale: number by number
        const bool single = !follows || now >= kScaleMax;
        if (works && !zero && now != was && !none) {
          const float k = clamp_scale(was) / now;
          u32x4* p = (u32x4*)codes;
          for (int i = w * 64 + lane; i < bs * D / 16; i += waves * 64) {
            u32x4 u = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = recode(u[j], k);
            p[i] = u;
          }
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // before others' codes go there
        }
        // the scale has been read, and what stood there is written, by all of the group
        if (waves > 1) __syncthreads();
        if (!works) continue;
        if (w == 0 && lane == 0) *scale = now;
        for (int tile = here; tile >= 0 && !single; tile -= waves) {   // the last is there
          if (tile != here) load(tile);
          if (none)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int j = 0; j < Quad<T>::W; ++j) v.raw[k][j] = u32x4{0, 0, 0, 0};
          const float by = none ? 1.0f : now;
          const int o = token_of(tile), d = dim_of(tile);
          const uint32_t at = part ? d * bs + o : o * D + d;
          if (inside(tile)) {
            if (part == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *(u32x2*)(codes + k * D + at) = u32x2{v.dims4(k, 0, by), v.dims4(k, 1, by)};
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) *(uint32_t*)(codes + i * bs + at) = v.tokens4(i, by);
            }
            continue;
          }
          // the run ends inside the tile
          if (part == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (o + k >= o0 && o + k < o0 + n)
                *(u32x2*)(codes + k * D + at) = u32x2{v.dims4(k, 0, by), v.dims4(k, 1, by)};
          } else {
            const bool whole = o >= o0 && o + 3 < o0 + n;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t u = v.tokens4(i, by);
              uint8_t* p = codes + i * bs + at;
              if (whole) *(uint32_t*)p = u;
              else
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (o + k >= o0 && o + k < o0 + n) p[k] = (uint8_t)(u >> (8 * k));
            }
          }
        }
        if (!single) continue;
        const float inv = none ? 1.0f : 1.0f / now;
        for (int j = 0; j < n; ++j) {      // one after the other: the later one stays
          const int o = a.slots[t + j] & (bs - 1);
          for (int i = w * 64 + lane; i < D; i += waves * 64) {
            const float f = (float)x[(t + j) * ld + i];
            codes[part ? i * bs + o : o * D + i] = to_code(none ? 0.0f : f * inv);
          }
        }
      }
    }
  }
}

}  // namespace

hipError_t run_tables(const TablesArgs& a, hipStream_t s) {
  // workgroups for the requests, and so many times them that a thread has four slots
  // and four entries, up to two a CU (1000 requests, a million slots: 128 in all 24 us,
  // 256 17; their blocks given back by 4 29 us, by 128 9 us)
  constexpr int64_t kMost = 512;
  const int64_t x = a.S < 256 * kTablesThreads ? (a.S + kTablesThreads - 1) / kTablesThreads : 256;
  const int64_t groups = x > 0 ? x : 1, each = 4 * kTablesThreads;
  const int64_t entries = (int64_t)a.S * a.max_blocks, work = a.T > entries ? a.T : entries;
  int64_t y = (work + groups * each - 1) / (groups * each);
  const int64_t most = kMost / groups > 1 ? kMost / groups : 1;
  y = y < 1 ? 1 : (y > most ? most : y);
  hipLaunchKernelGGL(tables_kernel, dim3((unsigned)groups, (unsigned)y), dim3(kTablesThreads), 0, s,
                     a);
  return hipGetLastError();
}

template <typename T>
hipError_t append_t(const AppendArgs& a, hipStream_t s) {
  // a wave a tile of 256 x 8 numbers, at most four a run
  const int tiles = a.block_size * a.dim / 2048;
  const int waves = tiles > 2 ? 4 : (tiles > 1 ? 2 : 1);
  const int items = a.heads * 2, per = 4 / waves, x = (items + per - 1) / per;
  // A workgroup looks at as many tokens as leave kAppendGroups workgroups, 64 at most: of
  // a prompt's tokens most do not begin a run, of single ones all do, one after the other
  // (8 heads of 128; one token a workgroup, this, 64 tokens: 2000 single tokens 31, 30 and
  // 173 us; 4004 tokens of 4 prompts 32, 10 and 13 us).
  constexpr int64_t kAppendGroups = 2048;
  int64_t tokens = (int64_t)a.T * x / kAppendGroups;
  tokens = tokens < 1 ? 1 : (tokens > 64 ? 64 : tokens);
  int64_t y = (a.T + tokens - 1) / tokens;
  if (y > 65535) y = 65535;
  const auto launch = [&](auto d) {
    constexpr int D = decltype(d)::value;
    hipLaunchKernelGGL((append_kernel<T, D>), dim3(x, (unsigned)y), dim3(256), 0, s, a, waves,
                       (int)tokens);
    return hipGetLastError();
  };
  if (a.dim == 64) return launch(std::integral_constant<int, 64>());
  if (a.dim == 128) return launch(std::integral_constant<int, 128>());
  return launch(std::integral_constant<int, 256>());
}

hipError_t run_append(const AppendArgs& a, hipStream_t s) {
  if (a.dtype == LIK_F16) return append_t<_Float16>(a, s);
  if (a.dtype == LIK_BF16) return append_t<__bf16>(a, s);
  return append_t<float>(a, s);
}

}  // namespace lik

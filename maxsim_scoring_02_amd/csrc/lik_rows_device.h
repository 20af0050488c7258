// Device-side building blocks of the row losses: 16-byte pieces of a row,
// softmax statistics and their merges, reductions over a wave.
//
// A row's exponentials are taken in base 2 relative to a maximum m:
//
//   e_c = 2^(z_c c - A),  c = scale log2(e),  A = fl(m c),  Z = sum_c e_c,
//
// one fused multiply-add and one v_exp_f32 per logit.  A is a rounded
// product, so every e_c carries the common factor 2^(mc - A); it cancels in
// q_c = e_c / Z, and the log-sum-exp takes it out again:
//
//   lse = scale m + ln2 (log2 Z - (mc - A)),  mc - A exact by one fma.
//
// Every wave takes its own maximum first and its exponentials relative to it,
// so that a row needs one meeting of its waves, where the pairs (m, Z) are
// merged.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "lik_rows_kernels.h"

namespace lik {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ---------------------------------------------------------------------------
// reductions over a wave: every lane gets the result, formed in one fixed tree
// ---------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_word(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(dpp_word<CTRL>(__float_as_uint(x)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint64_t lo = dpp_word<CTRL>((uint32_t)u), hi = dpp_word<CTRL>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(hi << 32 | lo));
}

// Both halves of x exchanged over 16 (or 32) lanes: a + b of the two results
// is x plus its partner's.
template <bool Wide>
__device__ __forceinline__ void swap_word(uint32_t x, uint32_t* a, uint32_t* b) {
  const auto r = Wide ? __builtin_amdgcn_permlane32_swap(x, x, false, false)
                      : __builtin_amdgcn_permlane16_swap(x, x, false, false);
  *a = r[0];
  *b = r[1];
}
template <bool Wide>
__device__ __forceinline__ void swap_half(float x, float* a, float* b) {
  uint32_t p, q;
  swap_word<Wide>(__float_as_uint(x), &p, &q);
  *a = __uint_as_float(p);
  *b = __uint_as_float(q);
}
template <bool Wide>
__device__ __forceinline__ void swap_half(double x, double* a, double* b) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  uint32_t p0, q0, p1, q1;
  swap_word<Wide>((uint32_t)u, &p0, &q0);
  swap_word<Wide>((uint32_t)(u >> 32), &p1, &q1);
  *a = __longlong_as_double((long long)((uint64_t)p1 << 32 | p0));
  *b = __longlong_as_double((long long)((uint64_t)q1 << 32 | q0));
}

struct MaxF {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumF {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a + b; }
};

// Every step's operands are the same two values in both partners, so all lanes
// hold the same bits at the end.
template <typename V, typename F>
__device__ __forceinline__ V wave_reduce(V v, F f) {
  v = f(v, dpp<0xB1>(v));     // quad_perm 1,0,3,2
  v = f(v, dpp<0x4E>(v));     // quad_perm 2,3,0,1
  v = f(v, dpp<0x141>(v));    // row_half_mirror: the other quad of eight
  v = f(v, dpp<0x140>(v));    // row_mirror: the other half of sixteen
  V a, b;
  swap_half<false>(v, &a, &b);
  v = f(a, b);
  swap_half<true>(v, &a, &b);
  return f(a, b);
}
__device__ __forceinline__ float wave_max(float v) { return wave_reduce(v, MaxF()); }
__device__ __forceinline__ float wave_sum(float v) { return wave_reduce(v, SumF()); }
__device__ __forceinline__ double wave_sum(double v) { return wave_reduce(v, SumF()); }

// The wave's number in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
}

// Threads that share LDS meet: one wave, or the workgroup.
template <int GT>
__device__ __forceinline__ void group_sync() {
  if constexpr (GT == 64) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// softmax statistics
// ---------------------------------------------------------------------------

// A row's softmax: e_c = exp2(fma(z_c, c, -A)), q_c = e_c / Z.
struct RowSoft {
  float m, c, A, Z;
};

// c and A from a maximum.  Up to |A| = 2^31 the factor 2^(mc - A) of A's rounding
// is at most 2^64, and sums of it stay in range.  From there on (rows of an empty
// document's -1e9 at a temperature, of the type's lowest values) logits that
// differ at all differ by 2^64 and more in their exponentials, so the power of two
// that brings m next to 2^64 serves as c: equal logits still give 1 and smaller
// ones 0.  An infinite m gives NaN throughout.
__device__ __forceinline__ RowSoft row_ref(float m, float scale) {
  RowSoft r;
  r.m = m;
  r.c = scale * kLog2e;
  r.A = m * r.c;
  if (!(fabsf(r.A) < 0x1p31f) && fabsf(m) < kInf) {
    r.c = ldexpf(1.0f, 64 - ilogbf(m));
    r.A = m * r.c;
  }
  r.Z = 0.0f;
  return r;
}

__device__ __forceinline__ float row_exp(const RowSoft& r, float z) {
  return exp2_fast(fmaf(z, r.c, -r.A));
}

// The reference of one part of a row (a wave, a piece).  A part without a
// finite logit has none: its exponentials of -inf are 0 there.
__device__ __forceinline__ RowSoft part_ref(float m, float scale) {
  RowSoft r = row_ref(m, scale);
  if (m == -kInf) r.A = 0.0f;
  return r;
}

// What a part's sum counts for in a row with the maximum s.m: 1 where the
// maxima are the same, nothing beside a maximum so large that only equal
// logits count.  The part's sum is relative to its A, the rounded product, so
// the product is rounded here too and never joined with the subtraction.
__device__ __forceinline__ float part_factor(const RowSoft& s, float m, float scale) {
#pragma clang fp contract(off)
  const float c = scale * kLog2e, A = m * c;
  if (m == s.m) return 1.0f;
  return s.c == c ? exp2_fast(A - s.A) : 0.0f;
}

// ln(Z 2^-(mc - A)), the log-sum-exp relative to the maximum.  The logarithm
// is split at the binary exponent, so its error stays near 2^-25 whatever Z.
__device__ __forceinline__ double row_ln_sum(const RowSoft& r) {
  int e;
  float f = frexpf(r.Z, &e);            // [0.5, 1)
  if (f < 0.70710678f) {
    f *= 2.0f;
    --e;
  }
  const double l2 = (double)e + (double)__builtin_amdgcn_logf(f) - (double)fmaf(r.m, r.c, -r.A);
  return kLn2 * l2;
}

// log softmax of one logit of the row
__device__ __forceinline__ double row_logp(const RowSoft& r, float z, float scale, double ln_sum) {
  return (double)scale * ((double)z - (double)r.m) - ln_sum;
}

// The parts (m, Z) of a row as one softmax, by one wave.  A row all of -inf has
// none: NaN.  With Part they are those of some of its columns, which may be.
template <bool Part = false>
__device__ __forceinline__ RowSoft merge_parts(const float2* __restrict__ parts, int n, float scale) {
  const int lane = threadIdx.x & 63;
  float m = -kInf;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, parts[i].x);
  RowSoft s = row_ref(wave_max(m), scale);
  float Z = 0.0f;
  for (int i = lane; i < n; i += 64) Z += parts[i].y * part_factor(s, parts[i].x, scale);
  s.Z = !Part && s.m == -kInf ? __builtin_nanf("") : wave_sum(Z);
  return s;
}

// The parts (m, Z) of a row as one softmax, by one lane.
__device__ __forceinline__ RowSoft lane_merge(const float2* __restrict__ part, int n, float scale) {
  constexpr int kAhead = 8;              // loads in flight; most rows have no more parts
  float2 x[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = i < n ? part[i] : make_float2(-kInf, 0.0f);
  float m = -kInf;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) m = fmaxf(m, x[i].x);
#pragma unroll 8
  for (int i = kAhead; i < n; ++i) m = fmaxf(m, part[i].x);
  RowSoft s = row_ref(m, scale);
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < n) s.Z += x[i].y * part_factor(s, x[i].x, scale);
#pragma unroll 8
  for (int i = kAhead; i < n; ++i) s.Z += part[i].y * part_factor(s, part[i].x, scale);
  if (m == -kInf) s.Z = __builtin_nanf("");
  return s;
}

// Sum over 256 threads, in every thread.
__device__ __forceinline__ double block_sum(double v, double* tmp) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) tmp[wave_id()] = v;
  __syncthreads();
  v = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------------------
// 16-byte pieces of a row
// ---------------------------------------------------------------------------

typedef uint32_t piece __attribute__((ext_vector_type(4)));
// rows start at any element, so pieces are loaded and stored at any alignment
typedef uint32_t piece_u2 __attribute__((ext_vector_type(4), aligned(2)));

template <typename T> struct PieceOf { static constexpr int N = 16 / sizeof(T); };

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(piece p, float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(p[i]);
  } else if constexpr (__is_same(T, __bf16)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(p[i] << 16);
      f[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)p[i]);
      f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(p[i] >> 16));
    }
  }
}

template <typename T>
__device__ __forceinline__ piece pack(const float* f) {
  if constexpr (sizeof(T) == 4) {
    return piece{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                 __float_as_uint(f[3])};
  } else {
    typedef T pair __attribute__((ext_vector_type(2)));
    piece p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __builtin_bit_cast(uint32_t, pair{(T)f[2 * i], (T)f[2 * i + 1]});
    return p;
  }
}

// Element c of a row piece below 4 GB: a 32-bit offset beside a scalar address.
template <typename T>
__device__ __forceinline__ T* at_column(T* p, int c) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
  return reinterpret_cast<T*>(reinterpret_cast<byte*>(p) + (uint32_t)c * (uint32_t)sizeof(T));
}

// -inf in every element
template <typename T>
__device__ __forceinline__ piece no_logits() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : (__is_same(T, __bf16) ? 0xff80ff80u : 0xfc00fc00u);
  return piece{w, w, w, w};
}

// Once: nothing reads the row again, so it need not stay in the caches.
template <bool Once, typename T>
__device__ __forceinline__ piece load_piece(const T* p) {
  const piece_u2* q = reinterpret_cast<const piece_u2*>(p);
  if constexpr (Once) return __builtin_nontemporal_load(q);
  return *q;
}
// far: past the caches.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, piece v, bool far) {
  piece_u2* q = reinterpret_cast<piece_u2*>(p);
  if (far) __builtin_nontemporal_store(v, q);
  else *q = v;
}

template <typename T>
__device__ __forceinline__ float piece_max(piece p, float m) {
  float f[PieceOf<T>::N];
  unpack<T>(p, f);
#pragma unroll
  for (int i = 0; i < PieceOf<T>::N; i += 2) m = max3(m, f[i], f[i + 1]);
  return m;
}

// Sum of N values in one fixed tree.
template <int N>
__device__ __forceinline__ float piece_total(const float* f) {
  float a = f[0], b = f[1];
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    a += f[i];
    b += f[i + 1];
  }
  return a + b;
}

// Waits for this wave's loads (and stores): vmcnt(0) alone.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// A uniform value that the compiler takes for a new one: comparisons with it are
// made where they are used and not kept in scalar registers from use to use.
__device__ __forceinline__ int opaque(int x) {
  x = __builtin_amdgcn_readfirstlane(x);
  asm("" : "+s"(x));
  return x;
}

// The same for a piece: what was unpacked of it is not kept for later.
__device__ __forceinline__ void opaque_piece(piece& p) { asm("" : "+v"(p)); }

// Elements before the first 16-byte boundary at or behind p, at most C.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int C) {
  const int h = (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T);
  return h < C ? h : C;
}

// How GT threads share `C` columns: a head up to a 16-byte boundary of what
// `at` points to and a tail behind the last whole piece, one column to a
// thread, and between them 16-byte pieces, dealt to the threads in turn.
template <typename T, int GT>
struct Deal {
  static constexpr int N = PieceOf<T>::N;
  int tid, head, pieces, edges;        // edges: columns of the head and the tail

  __device__ __forceinline__ Deal() {}
  __device__ __forceinline__ Deal(const T* at, int C, int t) {
    tid = t;
    head = head_of(at, C);
    pieces = (C - head) / N;
    edges = C - pieces * N;
  }
  __device__ __forceinline__ bool has(int i) const { return i * GT + tid < pieces; }
  __device__ __forceinline__ int column(int i) const { return head + (i * GT + tid) * N; }
  __device__ __forceinline__ bool has_edge() const { return tid < edges; }
  __device__ __forceinline__ int edge() const { return tid < head ? tid : tid + pieces * N; }
  // the thread that has column c
  __device__ __forceinline__ int owner(int c) const {
    const int p = c - head;
    const bool in = p >= 0 && p < pieces * N;
    return in ? p / N % GT : (p < 0 ? c : c - pieces * N);
  }
  __device__ __forceinline__ bool holds(int c) const { return owner(c) == tid; }
};

// The columns of a Deal on chip: an edge and NV pieces a thread at most in
// registers, NL more in LDS (at `lds`, NL * GT * 16 bytes, aligned to 16, for the
// rows that registers alone do not hold).  The pieces are aligned to
// the gradient's row where one is written (an unaligned store costs more than
// an unaligned load: 4096 x 131071 bf16 policy loss 508 us against 437), else to
// the logits'; with NL to the logits', which go to LDS directly.
template <typename T, int GT, int NV, bool Once = true, int NL = 0>
struct HeldRow {
  static constexpr int N = PieceOf<T>::N;
  static constexpr int64_t kColumns = (int64_t)GT * (NV + NL) * N;
  static constexpr int kLdsBytes = NL * GT * 16;
  Deal<T, GT> deal;
  piece d[NV];
  float edge;
  char* lds;

  // `grad`: where its gradient goes, or null
  __device__ __forceinline__ void load(const T* __restrict__ row, int C, int tid, const T* grad) {
    deal = Deal<T, GT>(grad && NL == 0 ? grad : row, C, tid);
    if constexpr (NL > 0) {
      // lane l's piece lands at the wave's base + 16 l
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (deal.has(NV + i))
          __builtin_amdgcn_global_load_lds(
              (const __attribute__((address_space(1))) void*)at_column(row, deal.column(NV + i)),
              (__attribute__((address_space(3))) void*)(lds + (i * (GT / 64) + wave_id()) * 1024),
              16, 0, Once ? 2 : 0);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      d[i] = no_logits<T>();
      if (deal.has(i)) d[i] = load_piece<Once>(at_column(row, deal.column(i)));
    }
    edge = -kInf;
    if (deal.has_edge()) edge = (float)row[deal.edge()];
  }
  __device__ __forceinline__ piece held(int i) const {
    if constexpr (NL > 0)
      if (i >= NV)
        return deal.has(i) ? *(const piece*)(lds + ((i - NV) * GT + deal.tid) * 16) : no_logits<T>();
    return d[i];
  }
  __device__ __forceinline__ float max() {
    float m = edge;
    const int pieces = opaque(deal.pieces);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * GT < pieces) m = piece_max<T>(d[i], m);
    if constexpr (NL > 0) {
      landed();
#pragma unroll
      for (int i = NV; i < NV + NL; ++i)
        if (i * GT < pieces) m = piece_max<T>(held(i), m);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) opaque_piece(d[i]);
    return m;
  }
  // LDS pieces are here (a wave reads back only what its own lanes loaded).
  __device__ __forceinline__ void landed() const {
    if constexpr (NL > 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  // Takes a column of this thread out of the row: -inf in its place.  After
  // landed().
  __device__ __forceinline__ void drop(int c) {
    const int p = c - deal.head, i = p / N / GT, j = p % N;
    if (p < 0 || p >= deal.pieces * N) {
      edge = -kInf;
      return;
    }
    const piece none = no_logits<T>();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (i == k) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t gone = w != j / (N / 4) ? 0u : N == 4 ? ~0u : 0xffffu << (j % 2 * 16);
          d[k][w] = (d[k][w] & ~gone) | (none[w] & gone);
        }
      }
    }
    if constexpr (NL > 0)
      if (i >= NV) reinterpret_cast<T*>(lds + ((i - NV) * GT + deal.tid) * 16)[j] = (T)-kInf;
  }
  __device__ __forceinline__ float sum(const RowSoft& s) {
    float z = row_exp(s, edge);
    const int pieces = opaque(deal.pieces);
#pragma unroll
    for (int i = 0; i < NV + NL; ++i) {
      if (i * GT < pieces) {
        float f[N];
        unpack<T>(held(i), f);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = row_exp(s, f[j]);
        z += piece_total<N>(f);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) opaque_piece(d[i]);
    return z;
  }
  // g = f(logit).  The pieces are all here by now; said once, before the stores,
  // it keeps the compiler from waiting for every store before the next piece.
  template <typename F>
  __device__ __forceinline__ void store(T* __restrict__ g, bool far, F f) const {
    wait_loads();
#pragma unroll
    for (int i = 0; i < NV + NL; ++i) {
      if (deal.has(i)) {
        float x[N];
        unpack<T>(held(i), x);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = f(x[j]);
        store_piece(at_column(g, deal.column(i)), pack<T>(x), far);
      }
    }
    if (deal.has_edge()) g[deal.edge()] = (T)f(edge);
  }
  __device__ __forceinline__ bool holds(int c) const { return deal.holds(c); }
};

// A constant over a row.
template <typename T, int GT>
__device__ __forceinline__ void fill_row(T* __restrict__ g, int C, int tid, float v) {
  constexpr int N = PieceOf<T>::N;
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = v;
  const piece p = pack<T>(f);
  const Deal<T, GT> deal(g, C, tid);
  for (int i = 0; deal.has(i); ++i) store_piece(at_column(g, deal.column(i)), p, false);
  if (deal.has_edge()) g[deal.edge()] = (T)v;
}

// The softmax of a group's columns: each wave's (m, Z), merged in LDS.  `tmp`
// holds two floats per wave.  With Part the columns are one part of a row, and
// one without a finite logit has Z = 0.  `meet` is done before the group meets.
struct Nothing {
  __device__ void operator()() const {}
};
template <int GT, bool Part = false, typename Held, typename F = Nothing>
__device__ __forceinline__ RowSoft held_softmax(Held& h, float scale, float* tmp,
                                                F meet = F()) {
  const RowSoft w = part_ref(wave_max(h.max()), scale);
  const float Z = wave_sum(h.sum(w));
  RowSoft s;
  meet();
  if constexpr (GT == 64) {
    s = row_ref(w.m, scale);
    s.Z = Z;
    group_sync<GT>();
  } else {
    constexpr int W = GT / 64;
    const int lane = threadIdx.x & 63;
    if (lane == 0) {
      tmp[2 * wave_id()] = w.m;
      tmp[2 * wave_id() + 1] = Z;
    }
    group_sync<GT>();
    const float m = lane < W ? tmp[2 * lane] : -kInf, z = lane < W ? tmp[2 * lane + 1] : 0.0f;
    s = row_ref(wave_max(m), scale);
    s.Z = wave_sum(z * part_factor(s, m, scale));
  }
  if (!Part && s.m == -kInf) s.Z = __builtin_nanf("");
  return s;
}

// ---------------------------------------------------------------------------
// grids
// ---------------------------------------------------------------------------

// A grid of n workgroups; linear_block() numbers them, those >= n are idle.
inline dim3 linear_grid(int64_t n) {
  const int64_t x = n < (1 << 20) ? n : (1 << 20);
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}
__device__ __forceinline__ int64_t linear_block() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// Groups of GT threads: workgroups of 256 threads at least.
template <int GT>
constexpr int group_threads() { return GT == 64 ? 256 : GT; }
template <int GT>
inline dim3 group_grid(int64_t R) { return linear_grid(GT == 64 ? (R + 3) / 4 : R); }
template <int GT>
__device__ __forceinline__ int64_t group_row() {
  return GT == 64 ? linear_block() * 4 + wave_id() : linear_block();
}
template <int GT>
__device__ __forceinline__ int group_tid() { return GT == 64 ? threadIdx.x & 63 : threadIdx.x; }

// The part of a row that a group of GT threads takes in a grid of `skip` and
// then R * n groups.
struct PartAt {
  int64_t r;
  int p, lo, cols;
};
template <int GT>
__device__ __forceinline__ PartAt part_at(const Parts& parts, int C, int skip) {
  PartAt x;
  const int64_t b = group_row<GT>() - skip;
  if constexpr (GT == 64) {              // whole rows
    x.r = b;
    x.p = x.lo = 0;
    x.cols = C;
    return x;
  }
  x.r = b / parts.n;
  x.p = (int)(b - x.r * parts.n);
  x.lo = x.p * parts.cols;
  x.cols = C - x.lo < parts.cols ? C - x.lo : parts.cols;
  return x;
}

// Calls f with the parts' group size as a constant.
template <typename F>
inline hipError_t parts_dispatch(const Parts& parts, F f) {
  if (parts.gt == 64) return f(std::integral_constant<int, 64>());
  return f(std::integral_constant<int, 256>());
}

// Policy loss of one row and its slope dl/dlogp.  x = logp - old, away =
// ref - logp (used with with_kl only).
__device__ __forceinline__ void policy_loss(float x, float adv, float low, float high, bool with_kl,
                                            float away, float kl, float* loss, float* slope) {
  const float rho = expf(x);
  // without an advantage 0, also where rho overflows; a NaN stays one
  const bool none = adv == 0.0f && rho == rho;
  const float u = none ? 0.0f : rho * adv;
  const float v = none ? 0.0f : fminf(fmaxf(rho, 1.0f - low), 1.0f + high) * adv;
  const bool flows = adv >= 0.0f ? rho <= 1.0f + high : rho >= 1.0f - low;
  float l = u != u ? u : -fminf(u, v);
  float g = flows || u != u ? -u : 0.0f;
  if (with_kl) {
    const float em1 = expm1f(away);
    // exp(d) - d - 1 cancels near 0: its series there.  Infinite at both ends (not inf - inf).
    const float d = away;
    const float series = d * d * (0.5f + d * (1.0f / 6 + d * (1.0f / 24 + d * (1.0f / 120 +
                         d * (1.0f / 720 + d * (1.0f / 5040 + d * (1.0f / 40320)))))));
    l += kl * (fabsf(d) < 0.5f ? series : em1 < kInf ? em1 - d : em1);
    g -= kl * em1;
  }
  *loss = l;
  *slope = g;
}

}  // namespace lik

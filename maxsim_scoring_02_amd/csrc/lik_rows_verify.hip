// Verification of drafted tokens (include/lik_rows.h, lik_verify_rows), in two
// launches.  The first looks at every row of target and drafter once and leaves the
// (m, Z) of its parts.  In the second a workgroup has a part of the row that its
// sequence ends at: it finds that row from the parts (every workgroup by itself, or a
// launch in between where they are many), sums the weights w of its columns, and the
// last of a sequence's workgroups to be done finds the part, and in it the column, that
// the random number points at.
// Weights are float32, sums of their pieces float64: a token of a vocabulary of 10^5
// has an interval of 10^-5 and less, which float32 sums would blur.
//
// 256 x 5 rows of 131072 bf16 (604 MB): the first launch is bound by reads, 6.9 TB/s, 87
// us; the rows of the ends take 6 us; the second reads the one or two rows that a sequence
// ends at again (134 MB at the most), 45 to 52 us.  Neither the reads (20 us at the first launch's
// rate) nor the exponentials (two a column, 7 us) explain that: its waves wait during
// 54% of their cycles, a part's sum, count and end one after the other.  One sequence of
// 5 rows of 32768: 3.8 and 11 us, latency: the second goes from offsets to drafts, to their
// logits, to the row's parts, to the sums and back into one part.
#include <hip/hip_runtime.h>

#include "lik_rows_device.h"
#include "lik_rows_kernels.h"

namespace lik {

namespace {

// Rows of a sequence, inside [0, R).
__device__ __forceinline__ void rows_of(const VerifyArgs& a, int64_t s, int64_t* lo, int64_t* hi) {
  const int64_t x = a.offsets[s], y = a.offsets[s + 1];
  *lo = x < 0 ? 0 : x;
  *hi = y > a.R ? a.R : y;
}

// Whether a sequence ends behind row r, or r lies in none.  Every wave looks for the
// first offset beyond r, in 64 places at a time.
__device__ __forceinline__ bool drafts_end(const VerifyArgs& a, int64_t r) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, n = a.S + 1;           // it is among offsets[lo .. lo + n]
  while (n > 0) {
    const int64_t step = (n + 63) / 64, i = lane * step;
    const int before = __popcll(__ballot(i < n && a.offsets[lo + (i < n ? i : 0)] <= r));
    if (before == 0) break;
    lo += (before - 1) * step + 1;
    n -= (before - 1) * step + 1;
    if (n > step - 1) n = step - 1;
  }
  return lo == 0 || lo > a.S || a.offsets[lo] == r + 1;
}

// Group b: a part of row b of the targets, then of the drafters.
template <typename T, int GT, bool Once>
__global__ __launch_bounds__(256) void verify_look_kernel(VerifyArgs a, Parts parts,
                                                          float2* __restrict__ out,
                                                          int* __restrict__ done) {
  __shared__ float tmp[2 * (GT / 64)];
  const int tid = group_tid<GT>();
  const int64_t threads = (int64_t)gridDim.x * gridDim.y * 256;
  for (int64_t s = linear_block() * 256 + threadIdx.x; s < a.S; s += threads) done[s] = 0;
  const PartAt at = part_at<GT>(parts, a.C, 0);
  const bool drafter = at.r >= a.R;
  const int64_t r = drafter ? at.r - a.R : at.r;
  if (r >= a.R || (drafter && !a.d)) return;
  if (drafter) {
    if (a.drafts[r] < 0 || drafts_end(a, r)) return;
  } else if (at.p == 0 && tid == 0) {
    a.tokens[r] = -1;
    a.logp[r] = 0.0f;
  }
  HeldRow<T, GT, kLookPieces, Once> h;
  h.load((drafter ? (const T*)a.d + r * a.draft_ld : (const T*)a.z + r * a.ld) + at.lo, at.cols, tid,
         nullptr);
  const RowSoft s = held_softmax<GT, true>(h, drafter ? a.draft_scale : a.scale, tmp);
  if (tid == 0) out[at.r * parts.n + at.p] = make_float2(s.m, s.Z);
}

// A row against its draft.
struct Outcome {
  RowSoft p, q;
  double ln_sum;
  bool more, broken, taken;
};
template <typename T>
__device__ __forceinline__ Outcome weigh(const VerifyArgs& a, const float2* mz, int n, int64_t r,
                                         int64_t hi) {
  Outcome v;
  const int x = a.drafts[r];
  v.more = r + 1 < hi && x >= 0;
  const bool in = v.more && x < a.C;
  const float zx = in ? (float)((const T*)a.z)[r * a.ld + x] : 0.0f;
  const float u = v.more ? a.accept_u[r] : 0.0f;
  v.p = merge_parts(mz + r * n, n, a.scale);
  v.q = v.p;
  double qx = 1.0;
  if (a.d && v.more) {
    const float dx = in ? (float)((const T*)a.d)[r * a.draft_ld + x] : 0.0f;
    v.q = merge_parts(mz + (a.R + r) * n, n, a.draft_scale);
    qx = in ? (double)row_exp(v.q, dx) / (double)v.q.Z : 0.0;
  }
  const double px = in ? (double)row_exp(v.p, zx) / (double)v.p.Z : 0.0;
  v.broken = v.p.Z != v.p.Z || v.q.Z != v.q.Z;
  v.taken = v.more && !v.broken && (double)u * qx < px;
  v.ln_sum = row_ln_sum(v.p);
  return v;
}

// The weights of a row's columns.
template <typename T>
struct Weights {
  const T *row, *drow;                   // drow: null without a drafter's row
  RowSoft p, q;
  float ip, iq;
  int x;                                 // a draft without a drafter's row, or -1

  __device__ __forceinline__ float of(float z, float d, int c) const {
    const float pc = row_exp(p, z) * ip;
    if (drow) return fmaxf(pc - row_exp(q, d) * iq, 0.0f);
    return c == x ? fmaxf(pc - 1.0f, 0.0f) : pc;
  }
};

constexpr int kVerifyPieces = 4;

// A part's weights by 256 threads, as 16-byte pieces of the row: sums a piece, the
// columns before the first and behind the last whole piece first and last.  The 4 or 8
// weights of a piece are added in float32: what that rounds is of the size of the weights'
// own error (in float64 1000 x 5 rows of 131072 553 us against 540, 256 x 5 149 against
// 147).
template <typename T, bool Once>
struct PartWeights {
  static constexpr int NV = kVerifyPieces, N = PieceOf<T>::N, kSlots = NV + 2;
  HeldRow<T, 256, NV, Once> z, d;

  __device__ __forceinline__ void load(const Weights<T>& w, int lo, int cols) {
    z.load(w.row + lo, cols, threadIdx.x, nullptr);
    if (w.drow) d.load(w.drow + lo, cols, threadIdx.x, w.row + lo);
  }
  // Weights of piece i in order.
  __device__ __forceinline__ void piece_of(const Weights<T>& w, int lo, int i, float* f) const {
    float g[N] = {};
    unpack<T>(z.d[i], f);
    if (w.drow) unpack<T>(d.d[i], g);
    const int c = lo + z.deal.column(i);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = w.of(f[j], g[j], c + j);
  }
  __device__ __forceinline__ float edge_of(const Weights<T>& w, int lo) const {
    return w.of(z.edge, w.drow ? d.edge : 0.0f, lo + z.deal.edge());
  }
  // This thread's sum in slot k.
  __device__ __forceinline__ double slot(const Weights<T>& w, int lo, int k) const {
    if (k == 0 || k == kSlots - 1) {
      const bool head = threadIdx.x < (unsigned)z.deal.head;
      return z.deal.has_edge() && head == (k == 0) ? (double)edge_of(w, lo) : 0.0;
    }
    if (!z.deal.has(k - 1)) return 0.0;
    float f[N];
    piece_of(w, lo, k - 1, f);
    return (double)piece_total<N>(f);
  }
  __device__ __forceinline__ int column_of(int k) const {
    return k == 0 || k == kSlots - 1 ? z.deal.edge() : z.deal.column(k - 1);
  }
};

// Sum over the lanes up to this one.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return v + __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lane_scan(double v) {
  v = dpp_add<0x111, 0xf>(v);            // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);            // the last of a row to the next
  return dpp_add<0x143, 0xc>(v);         // of the lower half to the upper
}
// v of lane k, the same for all lanes
__device__ __forceinline__ double lane_of(double v, int k) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, k);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), k);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// The column of a part at which the running sum passes `goal`; the last with a
// weight where rounding, or a goal beyond the part, leaves none.
template <typename T>
__device__ int pick(const Weights<T>& w, int lo, int cols, double goal, double* tmp, int* found) {
  typedef PartWeights<T, false> P;
  P part;
  part.load(w, lo, cols);
  const int lane = threadIdx.x & 63, wave = wave_id();
  double v[P::kSlots];
#pragma unroll
  for (int k = 0; k < P::kSlots; ++k) {
    v[k] = part.slot(w, lo, k);
    const double sum = wave_sum(v[k]);
    if (lane == 0) tmp[k * 4 + wave] = sum;
  }
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  double before = 0.0, at_before = 0.0;
  int at = -1, last = -1;
  for (int k = 0; k < P::kSlots * 4 && at < 0; ++k) {
    const double sum = tmp[k];
    if (sum > 0.0) last = k;
    if (before + sum > goal) {
      at = k;
      at_before = before;
    }
    before += sum;
  }
  const bool beyond = at < 0;
  if (beyond) at = last;
  if (at < 0) return -1;
  if (wave == at % 4) {
    const int k = at / 4;
    double mine = 0.0;
    float f[P::N] = {};
#pragma unroll
    for (int i = 0; i < P::kSlots; ++i)
      if (i == k) {
        mine = v[i];
        if (i > 0 && i < P::kSlots - 1) part.piece_of(w, lo, i - 1, f);
      }
    const double upto = at_before + lane_scan(mine);
    const uint64_t over = beyond ? 0 : __ballot(upto > goal), some = __ballot(mine > 0.0);
    const int who = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some | 1);
    if (lane == who) {
      int c = lo + part.column_of(k), hit = c;
      if (k > 0 && k < P::kSlots - 1) {
        double run = upto - mine;
        hit = -1;
        int positive = c;
#pragma unroll
        for (int j = 0; j < P::N; ++j) {
          run += (double)f[j];
          if (f[j] > 0.0f) positive = c + j;
          if (over && hit < 0 && run > goal) hit = c + j;
        }
        if (hit < 0) hit = positive;
      }
      *found = hit;
    }
  }
  __syncthreads();
  return *found;
}

// Where a sequence ends: the row a token is drawn from.
struct VerifyEnd {
  int64_t r;                             // -1: it has no rows
  double ln_sum;
  RowSoft p, q;
  int more, broken;
};

// Waits until this wave's stores have arrived; what follows stays behind them.
__device__ __forceinline__ void wait_stores() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

struct VerifySpace {
  float2* mz;                            // [2 R][parts of a row]
  double* sums;                          // [S][parts of a drawn row]
  int* done;                             // [S]
  VerifyEnd* ends;                       // [S], where they are found by a launch of their own
};

// The end of sequence s, by 256 threads: four rows at a time, a wave each, until one
// does not accept.  With `write` the outputs up to there too.
template <typename T>
__device__ __forceinline__ VerifyEnd find_end(const VerifyArgs& a, const float2* mz, int look,
                                              int64_t s, bool write) {
  __shared__ VerifyEnd rows[4];
  __shared__ int taken[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  VerifyEnd e;
  int64_t lo, hi;
  rows_of(a, s, &lo, &hi);
  if (hi <= lo) {
    if (write && tid == 0) a.accepted[s] = 0;
    e.r = -1;
    return e;
  }
  for (int64_t r0 = lo;; r0 += 4) {
    Outcome v;
    v.taken = false;
    const int64_t r = r0 + wave;
    if (r < hi) v = weigh<T>(a, mz, look, r, hi);
    if (lane == 0) {
      taken[wave] = r < hi && v.taken;
      if (r < hi) rows[wave] = VerifyEnd{r, v.ln_sum, v.p, v.q, v.more, v.broken};
    }
    __syncthreads();
    int w = 0;
    while (w < 4 && taken[w]) ++w;
    if (write && lane == 0 && wave < w) {
      const int x = a.drafts[r];
      a.tokens[r] = x;
      a.logp[r] = (float)row_logp(v.p, (float)((const T*)a.z)[r * a.ld + x], a.scale, v.ln_sum);
    }
    if (w < 4) {
      e = rows[w];
      break;
    }
    __syncthreads();
  }
  if (write && tid == 0) {
    a.accepted[s] = (int)(e.r - lo);
    if (e.broken) a.logp[e.r] = __builtin_nanf("");
  }
  return e;
}

template <typename T>
__global__ __launch_bounds__(256) void verify_end_kernel(VerifyArgs a, int look, VerifySpace ws) {
  const int64_t s = linear_block();
  if (s >= a.S) return;
  const VerifyEnd e = find_end<T>(a, ws.mz, look, s, true);
  if (threadIdx.x == 0) ws.ends[s] = e;
}

// Once: the rows are not in the cache behind the L2s, and go past it again.
// Found: by verify_end_kernel.
template <typename T, bool Once, bool Found>
__global__ __launch_bounds__(256) void verify_draw_kernel(VerifyArgs a, int look, Parts parts,
                                                          VerifySpace ws) {
  __shared__ double tmp[PartWeights<T, Once>::kSlots * 4];
  __shared__ int last, found;
  const int64_t s = linear_block() / parts.n;
  if (s >= a.S) return;
  const int part = (int)(linear_block() - s * parts.n);
  const int tid = threadIdx.x, lane = tid & 63;
  const VerifyEnd e = Found ? ws.ends[s] : find_end<T>(a, ws.mz, look, s, part == 0);
  const int64_t r = e.r;
  if (r < 0) return;
  const bool more = e.more, broken = e.broken;
  const double u = (double)a.sample_u[s];
  if (broken || u != u) return;
  Weights<T> w;
  w.row = (const T*)a.z + r * a.ld;
  w.drow = a.d && more ? (const T*)a.d + r * a.draft_ld : nullptr;
  w.p = e.p;
  w.q = e.q;
  w.ip = 1.0f / w.p.Z;
  w.iq = 1.0f / w.q.Z;
  w.x = !a.d && more ? a.drafts[r] : -1;
  const double ln_sum = e.ln_sum;
  const auto columns = [&](int p) {
    const int left = a.C - p * parts.cols;
    return left < parts.cols ? left : parts.cols;
  };
  double* sums = ws.sums + s * parts.n;
  if (parts.n > 1) {
    PartWeights<T, Once> mine;
    mine.load(w, part * parts.cols, columns(part));
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < PartWeights<T, Once>::kSlots; ++k) sum += mine.slot(w, part * parts.cols, k);
    sum = block_sum(sum, tmp);
    if (tid == 0) {
      // The sum goes past the caches by itself and has arrived when the count moves, for
      // which the wave waits: no cache is written back or dropped for it (with a fence of
      // the whole chip in each workgroup this launch took 435 us over 256 x 5 rows of
      // 131072).
      __hip_atomic_store(&sums[part], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      wait_stores();
      last = __hip_atomic_fetch_add(&ws.done[s], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             parts.n - 1;
    }
    __syncthreads();
    if (!last) return;
  }
  // the sequence's last workgroup: all of w, or all of p where nothing of it is left
  int token = -1;
  for (int pass = 0; token < 0 && pass < 2; ++pass) {
    double total = 0.0;
    if (pass == 1) {                     // p as it is
      w.drow = nullptr;
      w.x = -1;
    }
    if (pass == 1 || parts.n == 1) {
      // a part after the other, into the parts' places
      for (int p = 0; p < parts.n; ++p) {
        PartWeights<T, false> x;
        x.load(w, p * parts.cols, columns(p));
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < PartWeights<T, false>::kSlots; ++k) sum += x.slot(w, p * parts.cols, k);
        sum = block_sum(sum, tmp);
        if (tid == 0) __hip_atomic_store(&sums[p], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      wait_stores();                     // the other waves read them behind the meeting
      __syncthreads();
    }
    // every wave: a lane a part, 64 at a time
    const auto sum_at = [&](int p) {
      return p < parts.n
                 ? __hip_atomic_load(&sums[p], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                 : 0.0;
    };
    for (int p0 = 0; p0 < parts.n; p0 += 64) total += lane_of(lane_scan(sum_at(p0 + lane)), 63);
    if (!(total > 0.0)) continue;
    if (u < 0.0) {
      token = 0;
      break;
    }
    const double goal = u * total;
    double before = 0.0, at_before = 0.0, last_before = 0.0;
    int at = -1, some = -1;
    for (int p0 = 0; p0 < parts.n && at < 0; p0 += 64) {
      const double mine = sum_at(p0 + lane), upto = before + lane_scan(mine);
      const uint64_t over = __ballot(upto > goal && p0 + lane < parts.n);
      const uint64_t any = __ballot(mine > 0.0);
      if (any) {
        const int k = 63 - __builtin_clzll(any);
        some = p0 + k;
        last_before = k ? lane_of(upto, k - 1) : before;
      }
      if (over) {
        const int k = __builtin_ctzll(over);
        at = p0 + k;
        at_before = k ? lane_of(upto, k - 1) : before;
      }
      before = lane_of(upto, 63);
    }
    if (at < 0) {
      at = some;
      at_before = last_before;
    }
    __syncthreads();
    if (at < 0) break;
    token = pick(w, at * parts.cols, columns(at), goal - at_before, tmp, &found);
  }
  if (tid == 0 && token >= 0) {
    a.tokens[r] = token;
    a.logp[r] = (float)row_logp(w.p, (float)w.row[token], a.scale, ln_sum);
  }
}

template <typename T>
hipError_t verify_t(const VerifyArgs& a, char* ws, hipStream_t s) {
  const int64_t rows = a.d ? 2 * a.R : a.R;
  const Parts look = verify_look(a.R, a.C, a.dtype, a.d), draw = verify_draw(a.S, a.C, a.dtype);
  const VerifyLayout at = verify_layout(a.R, a.C, a.S, a.dtype, a.d);
  const VerifySpace space{(float2*)ws, (double*)(ws + at.sums), (int*)(ws + at.done),
                          (VerifyEnd*)(ws + at.ends)};
  const bool once = rows * a.C * elem_bytes_of(a.dtype) > kFarBytes;
  hipError_t e = parts_dispatch(look, [&](auto gt) {
    constexpr int GT = decltype(gt)::value;
    const auto kernel = once ? verify_look_kernel<T, GT, true> : verify_look_kernel<T, GT, false>;
    hipLaunchKernelGGL(kernel, group_grid<GT>(rows * look.n), dim3(256), 0, s, a, look, space.mz,
                       space.done);
    return hipGetLastError();
  });
  if (e != hipSuccess || a.S == 0) return e;
  const auto draws = [&](auto found) {
    constexpr bool F = decltype(found)::value;
    const auto kernel = once ? verify_draw_kernel<T, true, F> : verify_draw_kernel<T, false, F>;
    hipLaunchKernelGGL(kernel, linear_grid(a.S * draw.n), dim3(256), 0, s, a, look.n, draw, space);
  };
  if (a.S * draw.n > kVerifyEnds) {
    hipLaunchKernelGGL(verify_end_kernel<T>, linear_grid(a.S), dim3(256), 0, s, a, look.n, space);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    draws(std::true_type());
  } else {
    draws(std::false_type());
  }
  return hipGetLastError();
}

}  // namespace

hipError_t run_verify(const VerifyArgs& a, char* ws, hipStream_t s) {
  if (a.dtype == LIK_F16) return verify_t<_Float16>(a, ws, s);
  if (a.dtype == LIK_BF16) return verify_t<__bf16>(a, ws, s);
  return verify_t<float>(a, ws, s);
}

}  // namespace lik

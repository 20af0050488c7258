// Row losses whose gradient needs nothing beyond its own row: distillation
// from a teacher's top logits, and the clipped policy loss.
//
// Held rows (HeldRow): a group of threads loads its row once into registers,
// takes the statistics and writes the gradient from there, so the logits are
// read once and the gradient written once, which is all the traffic there is.
// One group a row: the rows on a CU are out of step, and one's loads overlap
// another's exponentials and stores.  (Groups that kept taking rows, with the
// next row's loads between the stores, were 4 to 25% slower.)
#include <hip/hip_runtime.h>

#include "lik_rows_device.h"
#include "lik_rows_kernels.h"

namespace lik {

namespace {

// loss = sum_r w_r l_r, rows of weight 0 left out.  One workgroup, so that the
// order is fixed; eight rows a thread are in flight at once.
__global__ __launch_bounds__(1024) void weighted_sum_kernel(const float* __restrict__ l,
                                                            const float* __restrict__ w, int64_t R,
                                                            float* __restrict__ loss) {
  __shared__ double tmp[16];
  double acc = 0.0;
  for (int64_t r0 = threadIdx.x; r0 < R; r0 += 8 * 1024) {
    float x[8], k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + i * 1024;
      x[i] = r < R ? l[r] : 0.0f;
      k[i] = r < R ? (w ? w[r] : 1.0f) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k[i] != 0.0f) acc += (double)k[i] * (double)x[i];
  }
  acc = wave_sum(acc);
  if ((threadIdx.x & 63) == 0) tmp[wave_id()] = acc;
  __syncthreads();
  acc = wave_sum((threadIdx.x & 63) < 16 ? tmp[threadIdx.x & 63] : 0.0);
  if (threadIdx.x == 0) *loss = (float)(w ? acc : acc / (double)R);
}

template <typename T>
struct PolicyArgs {
  const T* z;
  int64_t R, ld;
  int C;
  float scale;
  const int32_t* targets;
  const float *old_logp, *adv, *ref;
  float low, high, kl;
  const float* weight;
  float *row_loss, *logp;
  T* grad;
  int64_t gld;
  bool far;
};

// What a row's loss needs beside its softmax, loaded ahead of it.
struct PolicyRow {
  float zt, old, adv, ref, w;
};
template <typename T>
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs<T>& a, int64_t r, int t, float w) {
  const float zt = t < a.C ? (float)a.z[r * a.ld + t] : __builtin_nanf("");
  return PolicyRow{zt, a.old_logp[r], a.adv[r], a.ref ? a.ref[r] : 0.0f, w};
}
// Writes the row's loss and log-probability from one thread and returns the
// slope of w l along logp, times scale.
template <typename T>
__device__ __forceinline__ float policy_finish(const PolicyArgs<T>& a, int64_t r,
                                               const PolicyRow& x, const RowSoft& s, bool write) {
  const double lp = row_logp(s, x.zt, a.scale, row_ln_sum(s));
  float l, slope;
  policy_loss((float)(lp - (double)x.old), x.adv, a.low, a.high, a.ref != nullptr && a.kl != 0.0f,
              (float)((double)x.ref - lp), a.kl, &l, &slope);
  if (write) {
    a.row_loss[r] = l;
    a.logp[r] = (float)lp;
  }
  return x.w * slope * a.scale;
}

// Waves per SIMD that the held kernels' registers allow, with few pieces a
// thread and with many.
constexpr int held_waves(int nv, int few) { return nv <= 4 ? few : 4; }
constexpr int kPolicyWaves = 8, kDistillWaves = 6;

// Rows held on chip.  Bound by memory: 3584 read and 4096 written rows of 131072
// bf16 take 367 us, 5.5 TB/s, where a copy of that size runs at 4.9 to 5.2;
// 1024 x 32001 f32 45 us, 5.5 TB/s.  HBM traffic is the rows themselves (941 MB
// fetched, 1.07 GB written by the counters); VALU issue takes 67% of the cycles,
// but 15% fewer instructions did not change the time.
template <typename T, int GT, int NV, int NL>
__global__ __launch_bounds__(group_threads<GT>()) __attribute__((amdgpu_waves_per_eu(held_waves(NV, kPolicyWaves))))
void policy_held_kernel(const PolicyArgs<T> a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ float tmp[2 * (GT / 64)];
  const int64_t r = group_row<GT>();
  if (r >= a.R) return;
  const int tid = group_tid<GT>();
  const int t = a.targets[r];
  const float w = a.weight ? a.weight[r] : 1.0f / (float)a.R;
  T* g = a.grad + r * a.gld;
  if (t < 0 || w == 0.0f) {
    if (tid == 0) a.row_loss[r] = a.logp[r] = 0.0f;
    fill_row<T, GT>(g, a.C, tid, 0.0f);
    return;
  }
  HeldRow<T, GT, NV, true, NL> h;
  h.lds = lds;
  h.load(a.z + r * a.ld, a.C, tid, g);
  const PolicyRow x = policy_row(a, r, t, w);
  const RowSoft s = held_softmax<GT>(h, a.scale, tmp);
  const float k = policy_finish(a, r, x, s, tid == 0);
  const float kz = -k / s.Z;
  h.store(g, a.far, [&](float z) { return kz * row_exp(s, z); });
  // the same thread stored the column just before
  if (t < a.C && h.holds(t)) g[t] = (T)fmaf(kz, row_exp(s, x.zt), k);
}

// Rows in parts, the second look: the gradient, a workgroup a part.  For few
// rows the two looks are latency (61 x 100003 bf16: 5.3 and 7.5 us), for many
// rows too long to be held three passes over the row instead of two.
template <typename T>
__device__ __forceinline__ void policy_part(const PolicyArgs<T>& a, const PartAt& at,
                                            const float2* __restrict__ mz, int n) {
  const int64_t r = at.r;
  const int tid = threadIdx.x;
  const int t = a.targets[r];
  const float w = a.weight ? a.weight[r] : 1.0f / (float)a.R;
  T* g = a.grad + r * a.gld + at.lo;
  if (t < 0 || w == 0.0f) {
    fill_row<T, 256>(g, at.cols, tid, 0.0f);
    return;
  }
  HeldRow<T, 256, kGradPieces> h;
  h.load(a.z + r * a.ld + at.lo, at.cols, tid, g);
  const PolicyRow x = policy_row(a, r, t, w);
  const RowSoft s = merge_parts(mz + r * n, n, a.scale);
  const float k = policy_finish(a, r, x, s, false);
  const float kz = -k / s.Z;
  h.store(g, a.far, [&](float z) { return kz * row_exp(s, z); });
  const int c = t - at.lo;
  if (c >= 0 && c < at.cols && h.holds(c)) g[c] = (T)fmaf(kz, row_exp(s, x.zt), k);
}

// Losses and log-probabilities of the rows first, first + step, ..., a lane a
// row, and the thread's share of the weighted sum.
template <typename T>
__device__ __forceinline__ double policy_scalars(const PolicyArgs<T>& a, int64_t first, int64_t step,
                                                 const float2* __restrict__ mz, int n) {
  double acc = 0.0;
  for (int64_t r = first; r < a.R; r += step) {
    const int t = a.targets[r];
    const float w = a.weight ? a.weight[r] : 1.0f;
    if (t < 0 || w == 0.0f) {
      a.row_loss[r] = a.logp[r] = 0.0f;
      continue;
    }
    const PolicyRow x = policy_row(a, r, t, w);
    policy_finish(a, r, x, lane_merge(mz + r * n, n, a.scale), true);
    acc += (double)w * (double)a.row_loss[r];
  }
  return acc;
}

// Block 0: every row's loss and their sum, beside the others' gradient, so that
// few rows need no third launch.
constexpr int64_t kPolicyScalarRows = 1024;
template <typename T>
__global__ __launch_bounds__(256) void policy_parts_kernel(const PolicyArgs<T> a, Parts parts,
                                                           const float2* __restrict__ mz, int n,
                                                           float* __restrict__ loss) {
  __shared__ double tmp[4];
  if (linear_block() == 0) {
    const double acc = block_sum(policy_scalars(a, threadIdx.x, 256, mz, n), tmp);
    if (threadIdx.x == 0) *loss = (float)(a.weight ? acc : acc / (double)a.R);
    return;
  }
  const PartAt at = part_at<256>(parts, a.C, 1);
  if (at.r < a.R) policy_part(a, at, mz, n);
}

// Many rows: the scalars by a grid of their own.
template <typename T>
__global__ __launch_bounds__(256) void policy_scalars_kernel(const PolicyArgs<T> a,
                                                             const float2* __restrict__ mz, int n) {
  policy_scalars(a, linear_block() * 256 + threadIdx.x, a.R, mz, n);
}
template <typename T>
__global__ __launch_bounds__(256) void policy_grad_kernel(const PolicyArgs<T> a, Parts parts,
                                                          const float2* __restrict__ mz, int n) {
  const PartAt at = part_at<256>(parts, a.C, 0);
  if (at.r < a.R) policy_part(a, at, mz, n);
}

template <typename T>
struct DistillArgs {
  const T* z;
  int64_t R, ld;
  int C, K;
  float scale;
  const int32_t* idx;
  const float* val;
  const float* t_lse;
  const float* weight;
  float* row_loss;
  T* grad;
  int64_t gld;
  bool far;
};

// The teacher's list of one row in LDS.  Each thread has a chain of entries: those
// of the columns that a Deal gives to it, and in a kernel that has a part of the
// row others besides.  So a column's entries are all in one chain, and the thread
// that wrote a column's gradient can write it again without a meeting.
struct TeacherList {
  int32_t* col;        // column, -1 absent, | kAgain behind the column's first entry
  float* p;            // teacher logit, then its probability
  float* zs;           // the student's logit there
  int32_t* next;       // next entry of the chain, -1 at its end
  int* flags;          // 1: a column >= C, 4: an entry with mass
  int32_t* head;       // first entry of each thread's chain
};
constexpr int32_t kAgain = 1 << 24;
static_assert(kDistillMaxC < kAgain, "a column and its mark share a word");

__device__ __forceinline__ TeacherList teacher_at(char* p, int K) {
  TeacherList L;
  L.col = (int32_t*)p;
  L.p = (float*)p + K;
  L.zs = (float*)p + 2 * K;
  L.next = (int32_t*)p + 3 * K;
  L.flags = (int*)p + 4 * K;
  L.head = (int32_t*)p + 4 * K + 1;
  return L;
}
__device__ __forceinline__ int entry_col(int32_t c) { return c & (kAgain - 1); }

// The columns that a kernel's group has, from lo on, shared by `deal`, and the
// chain of any column.
template <typename T, int GT>
struct TeacherAt {
  Deal<T, GT> deal;
  int lo, cols;
  __device__ __forceinline__ bool has(int j) const { return j >= lo && j - lo < cols; }
  __device__ __forceinline__ int chain(int j) const {
    return has(j) ? deal.owner(j - lo) : j & (GT - 1);
  }
};

// One entry of the list into LDS, without the student's logit.
template <typename T, int GT>
__device__ __forceinline__ void teacher_entry(const DistillArgs<T>& a, const TeacherList& L,
                                              const TeacherAt<T, GT>& at, int k, int32_t j, float t) {
  const bool in = j >= 0 && j < a.C;
  int flags = j >= a.C ? 1 : 0;
  if (in) {
    if (t != -kInf) flags |= 4;
    L.next[k] = atomicExch(&L.head[at.chain(j)], k);
  }
  L.col[k] = in ? j : -1;
  L.p[k] = t;
  if (flags) atomicOr(L.flags, flags);
}

// Marks what is listed a second time, by one wave: a column's first entry stands
// for it.  The order within the chains does not matter.
template <typename T, int GT>
__device__ __forceinline__ bool teacher_again(const TeacherList& L, const TeacherAt<T, GT>& at,
                                              int K, int lane) {
  bool any = false;
  for (int k = lane; k < K; k += 64) {
    const int32_t c = L.col[k];
    if (c < 0) continue;
    bool again = false;
    for (int i = L.head[at.chain(c)]; i >= 0; i = L.next[i])
      if (i < k) again |= entry_col(L.col[i]) == c;
    if (again) L.col[k] = c | kAgain;
    any |= again;
  }
  return __any(any);
}

// A thread's first entry, loaded ahead of the row, and the student's logit there,
// loaded behind it: loads come back in order, so what needs the entry does not
// wait for the row, and the logit is not asked for before the row is there.
template <typename T>
struct TeacherAhead {
  int32_t j = -1;
  float t = 0.0f, z = 0.0f;
  __device__ __forceinline__ void entry(const DistillArgs<T>& a, int64_t r, int tid) {
    if (tid < a.K) {
      j = a.idx[r * a.K + tid];
      t = a.val[r * a.K + tid];
    }
  }
  __device__ __forceinline__ void logit(const DistillArgs<T>& a, const T* row) {
    if (j >= 0 && j < a.C) z = (float)row[j];
  }
};

// The list into LDS; returns the flags.
template <typename T, int GT>
__device__ __forceinline__ int teacher_fill(const DistillArgs<T>& a, const TeacherList& L,
                                            int64_t r, int tid, const TeacherAhead<T>& x,
                                            const TeacherAt<T, GT>& at) {
  L.head[tid] = -1;
  if (tid == 0) *L.flags = 0;
  group_sync<GT>();
  if (tid < a.K) teacher_entry(a, L, at, tid, x.j, x.t);
  for (int k = tid + GT; k < a.K; k += GT)
    teacher_entry(a, L, at, k, a.idx[r * a.K + k], a.val[r * a.K + k]);
  group_sync<GT>();
  return *L.flags;
}

// What the list adds up to.  One wave goes over it (every wave doing so for
// itself, without LDS between them, cost 2% of 4096 rows of 65536 and 131072 bf16
// with 64 entries): first, while the row is on its way, the teacher's side ...
struct TeacherSums {
  double mass;        // teacher probability of the list
  double terms;       // sum p (log p - scale (z - base))
  float base;         // m, or 0 where that is infinite
  float m, Z;         // the listed columns as a part of the student's row
  int columns;        // how many those are
  bool again;         // a column is listed twice
};
__device__ __forceinline__ void teacher_probs(const TeacherList& L, int K, float scale,
                                                const float* t_lse, TeacherSums* x, int lane) {
  double lt;
  if (t_lse) {
    lt = (double)*t_lse;
  } else {
    float m = -kInf, sum = 0.0f;
    for (int k = lane; k < K; k += 64)
      if (L.col[k] >= 0) m = fmaxf(m, L.p[k]);
    m = wave_max(m);
    for (int k = lane; k < K; k += 64)
      if (L.col[k] >= 0) sum += expf(scale * (L.p[k] - m));
    lt = (double)scale * (double)m + (double)logf(wave_sum(sum));
  }
  x->mass = x->terms = 0.0;
  for (int k = lane; k < K; k += 64) {
    const float t = L.p[k];
    const double lp = (double)scale * (double)t - lt;
    const float p = L.col[k] < 0 || t == -kInf ? 0.0f : expf((float)lp);
    L.p[k] = p;
    x->mass += (double)p;
    if (p != 0.0f) x->terms += (double)p * lp;
  }
}
// ... then the student's.  The same wave; sums in its lane 0.
template <typename T>
__device__ __forceinline__ void teacher_sums(const DistillArgs<T>& a, const TeacherList& L,
                                             const T* row, float z0, TeacherSums* x, int lane) {
  float m = -kInf;
#pragma unroll 4
  for (int k = lane; k < a.K; k += 64) {
    const int32_t c = L.col[k];
    float z = z0;
    if (k >= 64) z = c >= 0 ? (float)row[entry_col(c)] : 0.0f;
    L.zs[k] = z;
    if (c >= 0) m = fmaxf(m, z);
  }
  const RowSoft s = part_ref(wave_max(m), a.scale);
  // logits next to float32's ends are told apart only relative to each other
  x->base = fabsf(s.m) < kInf ? s.m : 0.0f;
  float Z = 0.0f;
  int columns = 0;
  for (int k = lane; k < a.K; k += 64) {
    const int32_t c = L.col[k];
    const float z = L.zs[k], p = L.p[k];
    if (p != 0.0f) x->terms -= (double)p * ((double)a.scale * ((double)z - (double)x->base));
    if (c >= 0 && !(c & kAgain)) {
      Z += row_exp(s, z);
      ++columns;
    }
  }
  x->mass = wave_sum(x->mass);
  x->terms = wave_sum(x->terms);
  x->m = s.m;
  x->Z = wave_sum(Z);
  x->columns = (int)wave_sum((float)columns);      // at most 1024: exact
}

// Loss of a row and its gradient: k = w scale,
//   on * e - k p    on listed columns, e as in `row`, the softmax of all columns
//   off * e         on the others, e as in `others`: theirs where the rest has a
//                   term (so that they are told apart however far below the
//                   listed ones they lie), else the row's
struct DistillRow {
  float loss, on, off;
  RowSoft row, others;
};
// s: the softmax of all columns, or with_rest of those not listed.
__device__ __forceinline__ DistillRow distill_row(const TeacherSums& x, bool with_rest, int C,
                                                  float scale, float k, const RowSoft& s) {
  DistillRow d;
  d.row = d.others = s;
  if (with_rest) {
    if (s.m == -kInf) d.others.A = 0.0f;                // every e is 0
    d.row = row_ref(fmaxf(s.m, x.m), scale);
    d.row.Z = s.Z * part_factor(d.row, s.m, scale);
    if (x.columns) d.row.Z += x.Z * part_factor(d.row, x.m, scale);
  }
  if (d.row.m == -kInf) d.row.Z = __builtin_nanf("");
  const double ln_sum = row_ln_sum(d.row);
  // log q = scale (z - m) - ln_sum, so sum p (log p - log q) is
  double l = x.terms;
  if (x.mass != 0.0)
    l += x.mass * ((double)scale * ((double)d.row.m - (double)x.base) + ln_sum);
  const float M = (float)x.mass;
  d.on = d.off = k * (M / d.row.Z);
  if (with_rest && x.columns < C) {
    const float p = x.mass != x.mass ? __builtin_nanf("") : (float)fmax(0.0, 1.0 - x.mass);
    // sum p (log p - log q) over the rest; q is 0 where no column is finite, and
    // ln_sum NaN where none of the whole row is
    if (p != 0.0f)
      l += (double)p * ((double)logf(p) - (s.Z == 0.0f ? -(double)kInf - ln_sum
                                                       : row_logp(d.row, s.m, scale, ln_sum) +
                                                             row_ln_sum(s)));
    const float all = (float)(x.mass + (double)p);
    d.on = k * (all / d.row.Z);
    d.off = d.on * part_factor(d.row, s.m, scale) - (s.Z == 0.0f ? 0.0f : k * (p / s.Z));
  }
  d.loss = (float)l;
  return d;
}

// The gradient on the listed columns, over what the same thread wrote there with
// the row.
__device__ __forceinline__ float teacher_grad(const TeacherList& L, int K, int k, const RowSoft& s,
                                              float on, float weight, bool again) {
  double p = (double)L.p[k];
  if (again)
    for (int j = k + 1; j < K; ++j)
      if (L.col[j] == (L.col[k] | kAgain)) p += (double)L.p[j];
  return on * row_exp(s, L.zs[k]) - weight * (float)p;
}
template <typename T, int GT>
__device__ __forceinline__ void teacher_grads(const TeacherList& L, const TeacherAt<T, GT>& at,
                                              int K, const RowSoft& s, float on, float weight,
                                              bool again, T* __restrict__ g) {
  for (int k = L.head[at.deal.tid]; k >= 0; k = L.next[k]) {
    const int32_t c = L.col[k];
    if (!(c & kAgain) && at.has(c)) g[c] = (T)teacher_grad(L, K, k, s, on, weight, again);
  }
}

// Rows held on chip.  4096 x 65536 bf16 with 64 entries a row and the rest's term:
// 208 to 220 us, 4.9 to 5.2 TB/s, a call 221 us (without the rest 219), 11% behind
// the policy loss on the same rows (198): the list costs meetings and LDS passes in
// a row's life, and the listed columns' second stores 2%.  4096 x 131072 f32, partly
// in LDS, 930 us a call, 4.6 TB/s (in parts 1675).
template <typename T, int GT, int NV, int NL>
__global__ __launch_bounds__(group_threads<GT>()) __attribute__((amdgpu_waves_per_eu(held_waves(NV, kDistillWaves))))
void distill_held_kernel(const DistillArgs<T> a) {
  __shared__ float tmp[2 * (GT / 64)];
  __shared__ TeacherSums sums[GT == 64 ? 4 : 1];
  extern __shared__ __attribute__((aligned(16))) char lists[];
  const int64_t r = group_row<GT>();
  if (r >= a.R) return;
  const int tid = group_tid<GT>(), lane = threadIdx.x & 63;
  const int group = GT == 64 ? wave_id() : 0;
  const bool counts = GT == 64 || wave_id() == 0;          // the wave that goes over the list
  const float w = a.weight ? a.weight[r] : 1.0f / (float)a.R;
  T* g = a.grad + r * a.gld;
  if (w == 0.0f) {
    if (tid == 0) a.row_loss[r] = 0.0f;
    fill_row<T, GT>(g, a.C, tid, 0.0f);
    return;
  }
  const T* row = a.z + r * a.ld;
  TeacherAhead<T> ahead;
  ahead.entry(a, r, tid);
  HeldRow<T, GT, NV, true, NL> h;
  h.lds = lists;
  const TeacherList L = teacher_at(lists + h.kLdsBytes + group * teacher_bytes(a.K, GT), a.K);
  h.load(row, a.C, tid, g);
  if (counts) ahead.logit(a, row);
  const TeacherAt<T, GT> at{h.deal, 0, a.C};
  const int flags = teacher_fill(a, L, r, tid, ahead, at);
  const bool with_rest = a.t_lse != nullptr;
  if (!with_rest && !(flags & 5)) {
    // no entry with mass
    h.landed();                         // before the LDS goes to another group
    if (tid == 0) a.row_loss[r] = 0.0f;
    fill_row<T, GT>(g, a.C, tid, 0.0f);
    return;
  }
  TeacherSums x;
  if (counts) {
    x.again = teacher_again(L, at, a.K, lane);
    teacher_probs(L, a.K, a.scale, with_rest ? a.t_lse + r : nullptr, &x, lane);
  }
  if (with_rest) {
    h.landed();
    for (int k = L.head[tid]; k >= 0; k = L.next[k]) h.drop(entry_col(L.col[k]));
  }
  const RowSoft s = held_softmax<GT, true>(h, a.scale, tmp, [&] {
    if (!counts) return;
    teacher_sums(a, L, row, ahead.z, &x, lane);
    if (lane == 0) sums[group] = x;
  });
  const float k = w * a.scale + (flags & 1 ? __builtin_nanf("") : 0.0f);
  const DistillRow d = distill_row(sums[group], with_rest, a.C, a.scale, k, s);
  if (tid == 0) a.row_loss[r] = flags & 1 ? __builtin_nanf("") : d.loss;
  h.store(g, a.far, [&](float z) { return d.off * row_exp(d.others, z); });
  teacher_grads(L, at, a.K, d.row, d.on, k, sums[group].again, g);
}

// Rows in parts, the first look: each part's (m, Z), listed columns left out
// where the rest has a term of its own.  256 threads a part however short the row
// and loads through the caches, also where no gradient follows: without one
// 65536 x 300 f32 (16 entries) takes 244 us, with it, held, 90; 4096 x 100003 bf16
// 157 us, the same rows' log-probabilities 111.
template <typename T>
__global__ __launch_bounds__(256) void distill_stats_kernel(const DistillArgs<T> a, Parts parts,
                                                            float2* __restrict__ mz) {
  __shared__ float tmp[8];
  __shared__ int32_t head[256], next[kDistillMaxK], col[kDistillMaxK];
  const PartAt at = part_at<256>(parts, a.C, 0);
  if (at.r >= a.R) return;
  const int64_t r = at.r;
  const int tid = threadIdx.x;
  if (a.weight && a.weight[r] == 0.0f) return;
  HeldRow<T, 256, kLookPieces, false> h;
  h.load(a.z + r * a.ld + at.lo, at.cols, tid, nullptr);
  const bool with_rest = a.t_lse != nullptr;
  if (with_rest) {
    head[tid] = -1;
    __syncthreads();
    for (int k = tid; k < a.K; k += 256) {
      const int64_t c = (int64_t)a.idx[r * a.K + k] - at.lo;
      if (c < 0 || c >= at.cols) continue;
      col[k] = (int)c;
      next[k] = atomicExch(&head[h.deal.owner((int)c)], k);
    }
    __syncthreads();
    for (int k = head[tid]; k >= 0; k = next[k]) h.drop(col[k]);
  }
  const RowSoft s = held_softmax<256, true>(h, a.scale, tmp);
  if (tid == 0) mz[r * parts.n + at.p] = make_float2(s.m, s.Z);
}

// The second look: loss (part 0) and gradient.
template <typename T>
__global__ __launch_bounds__(256) void distill_parts_kernel(const DistillArgs<T> a, Parts parts,
                                                            const float2* __restrict__ mz, int n) {
  __shared__ TeacherSums sums;
  extern __shared__ __attribute__((aligned(16))) char lists[];
  const PartAt part = part_at<256>(parts, a.C, 0);
  if (part.r >= a.R) return;
  const int64_t r = part.r;
  const int tid = threadIdx.x;
  const float w = a.weight ? a.weight[r] : 1.0f / (float)a.R;
  const bool first = part.p == 0 && tid == 0;
  T* g = a.grad ? a.grad + r * a.gld : nullptr;
  if (!g && part.p != 0) return;
  if (w == 0.0f) {
    if (first) a.row_loss[r] = 0.0f;
    if (g) fill_row<T, 256>(g + part.lo, part.cols, tid, 0.0f);
    return;
  }
  const T* row = a.z + r * a.ld;
  const TeacherList L = teacher_at(lists, a.K);
  TeacherAhead<T> ahead;
  ahead.entry(a, r, tid);
  if (wave_id() == 0) ahead.logit(a, row);
  HeldRow<T, 256, kGradPieces> h;
  if (g) h.load(row + part.lo, part.cols, tid, g + part.lo);
  else h.deal = Deal<T, 256>(row + part.lo, part.cols, tid);
  const TeacherAt<T, 256> at{h.deal, part.lo, part.cols};
  const int flags = teacher_fill(a, L, r, tid, ahead, at);
  const bool with_rest = a.t_lse != nullptr;
  if (!with_rest && !(flags & 5)) {
    if (first) a.row_loss[r] = 0.0f;
    if (g) fill_row<T, 256>(g + part.lo, part.cols, tid, 0.0f);
    return;
  }
  if (wave_id() == 0) {
    TeacherSums x;
    x.again = teacher_again(L, at, a.K, tid);
    teacher_probs(L, a.K, a.scale, with_rest ? a.t_lse + r : nullptr, &x, tid);
    teacher_sums(a, L, row, ahead.z, &x, tid);
    if (tid == 0) sums = x;
  }
  const RowSoft s = merge_parts<true>(mz + r * n, n, a.scale);
  __syncthreads();
  const float k = w * a.scale + (flags & 1 ? __builtin_nanf("") : 0.0f);
  const DistillRow d = distill_row(sums, with_rest, a.C, a.scale, k, s);
  if (first) a.row_loss[r] = flags & 1 ? __builtin_nanf("") : d.loss;
  if (g) {
    h.store(g + part.lo, a.far, [&](float z) { return d.off * row_exp(d.others, z); });
    teacher_grads(L, at, a.K, d.row, d.on, k, sums.again, g);
  }
}

// Calls f with the group size, the pieces per thread in registers and those in
// LDS that hold C columns.  bf16, us a call of the policy loss / of distillation with
// 64 entries a row / and with the rest's term:
//   16384 x 4096    one wave 56 / 77 / 78, 256 threads 56 / 93 / 103
//   8192 x 8192     one wave 53 / 69 / 73, 256 threads 51 / 64 / 70
//   4096 x 32768    256 threads 93 / 102 / 106, 512 threads 90 / 100 / 102
//   4096 x 65536    256 threads 253 / 338 / 346, 512 threads 198 / 219 / 221,
//                   1024 threads 200 / 269 / 288
template <typename T, typename F>
hipError_t held_dispatch(int64_t C, F f) {
#define LIK_HELD(GT, NV, NL)                                                     \
  if (C <= HeldRow<T, GT, NV, true, NL>::kColumns)                               \
    return f(std::integral_constant<int, GT>(), std::integral_constant<int, NV>(), \
             std::integral_constant<int, NL>());
  LIK_HELD(64, 4, 0)
  LIK_HELD(64, 8, 0)
  LIK_HELD(256, 4, 0)
  LIK_HELD(256, 8, 0)
  LIK_HELD(512, 8, 0)
  LIK_HELD(512, 16, 0)
  LIK_HELD(1024, 16, 0)
  LIK_HELD(1024, 23, 9)
#undef LIK_HELD
  return hipErrorInvalidValue;
}

// Allows a kernel `most` bytes of LDS where this call's are more than it has by
// default; asking again costs little beside so large a row.
template <typename K>
hipError_t allow_lds(K kernel, size_t bytes, size_t most) {
  if (bytes <= kDefaultLds) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

hipError_t weighted_sum(const float* l, const float* w, int64_t R, float* loss, hipStream_t s) {
  hipLaunchKernelGGL(weighted_sum_kernel, dim3(1), dim3(1024), 0, s, l, w, R, loss);
  return hipGetLastError();
}

template <typename T>
hipError_t policy_t(const Rows& a, const int32_t* targets, const float* old_logp, const float* adv,
                    const float* ref, float low, float high, float kl, const float* weight,
                    float* row_loss, float* logp, float* loss, char* ws, hipStream_t s) {
  const PolicyArgs<T> p{(const T*)a.z, a.R, a.ld, (int)a.C, a.scale, targets, old_logp, adv, ref,
                        low, high, kl, weight, row_loss, logp, (T*)a.grad, a.grad_ld, a.far()};
  if (a.grad && rows_held(a.R, a.C, a.dtype, kHeldBytes)) {
    const hipError_t e = held_dispatch<T>(a.C, [&](auto gt, auto nv, auto nl) {
      constexpr int GT = decltype(gt)::value, NV = decltype(nv)::value, NL = decltype(nl)::value;
      constexpr size_t lds = HeldRow<T, GT, NV, true, NL>::kLdsBytes;
      const hipError_t e = allow_lds(policy_held_kernel<T, GT, NV, NL>, lds, lds);
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((policy_held_kernel<T, GT, NV, NL>), group_grid<GT>(a.R),
                         dim3(group_threads<GT>()), lds, s, p);
      return hipGetLastError();
    });
    return e != hipSuccess ? e : weighted_sum(row_loss, weight, a.R, loss, s);
  }
  const Parts look = look_parts(a.R, a.C, a.dtype);
  const Parts parts = grad_parts(a.R, a.C, a.dtype);
  const int64_t n_parts = a.grad ? a.R * parts.n : 0;
  float2* mz = (float2*)ws;
  hipError_t e = run_parts(a, look, targets, weight, nullptr, 0, mz, s);
  if (e != hipSuccess) return e;
  if (a.R <= kPolicyScalarRows) {
    hipLaunchKernelGGL(policy_parts_kernel<T>, linear_grid(n_parts + 1), dim3(256), 0, s, p, parts,
                       mz, look.n, loss);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(policy_scalars_kernel<T>, linear_grid((a.R + 255) / 256), dim3(256), 0, s, p,
                     mz, look.n);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (n_parts) {
    hipLaunchKernelGGL(policy_grad_kernel<T>, linear_grid(n_parts), dim3(256), 0, s, p, parts, mz,
                       look.n);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return weighted_sum(row_loss, weight, a.R, loss, s);
}

template <typename T>
hipError_t distill_t(const Rows& a, const int32_t* idx, const float* val, int64_t K,
                     const float* t_lse, const float* weight, float* row_loss, char* ws,
                     hipStream_t s) {
  const DistillArgs<T> p{(const T*)a.z, a.R, a.ld, (int)a.C, (int)K, a.scale, idx, val, t_lse,
                         weight, row_loss, (T*)a.grad, a.grad_ld, a.far()};
  if (a.grad && rows_held(a.R, a.C, a.dtype, K > kDistillLdsK ? kRegisterBytes : kHeldBytes))
    return held_dispatch<T>(a.C, [&](auto gt, auto nv, auto nl) {
      constexpr int GT = decltype(gt)::value, NV = decltype(nv)::value, NL = decltype(nl)::value;
      static_assert(HeldRow<T, GT, NV, true, NL>::kLdsBytes == NL * GT * 16, "distill_lds");
      const size_t lds = distill_lds(K, GT, NL);
      const hipError_t e =
          allow_lds(distill_held_kernel<T, GT, NV, NL>, lds, distill_lds_most(GT, NL));
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((distill_held_kernel<T, GT, NV, NL>), group_grid<GT>(a.R),
                         dim3(group_threads<GT>()), lds, s, p);
      return hipGetLastError();
    });
  const Parts look = look_parts(a.R, a.C, a.dtype);
  const Parts parts = a.grad ? grad_parts(a.R, a.C, a.dtype) : Parts{(int)a.C, 1, 256};
  float2* mz = (float2*)ws;
  hipLaunchKernelGGL(distill_stats_kernel<T>, linear_grid(a.R * look.n), dim3(256), 0, s, p, look,
                     mz);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  static_assert(teacher_bytes(kDistillMaxK, 256) <= kDefaultLds, "never has to be allowed");
  hipLaunchKernelGGL(distill_parts_kernel<T>, linear_grid(a.R * parts.n), dim3(256),
                     teacher_bytes(K, 256), s, p, parts, mz, look.n);
  return hipGetLastError();
}

}  // namespace

hipError_t run_policy(const Rows& a, const int32_t* targets, const float* old_logp,
                      const float* adv, const float* ref, float low, float high, float kl,
                      const float* weight, float* row_loss, float* logp, float* loss, char* ws,
                      hipStream_t s) {
  const auto run = a.dtype == LIK_F16    ? policy_t<_Float16>
                   : a.dtype == LIK_BF16 ? policy_t<__bf16>
                                         : policy_t<float>;
  return run(a, targets, old_logp, adv, ref, low, high, kl, weight, row_loss, logp, loss, ws, s);
}

hipError_t run_distill(const Rows& a, const int32_t* idx, const float* val, int64_t K,
                       const float* t_lse, const float* weight, float* row_loss, float* loss,
                       char* ws, hipStream_t s) {
  const auto run = a.dtype == LIK_F16    ? distill_t<_Float16>
                   : a.dtype == LIK_BF16 ? distill_t<__bf16>
                                         : distill_t<float>;
  const hipError_t e = run(a, idx, val, K, t_lse, weight, row_loss, ws, s);
  return e != hipSuccess ? e : weighted_sum(row_loss, weight, a.R, loss, s);
}

}  // namespace lik

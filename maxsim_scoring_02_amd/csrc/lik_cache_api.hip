// C ABI of the 8-bit cache (include/lik_cache.h): argument checks and dispatch.
#include <hip/hip_runtime.h>

#include "lik.h"
#include "lik_cache.h"
#include "lik_cache_kernels.h"
#include "lik_host.h"

namespace {

using lik::aligned16;
using lik::aligned4;
using lik::check_device;
using lik::fail;
using lik::mul_ok;
using lik::ok;
using lik::Span;

lik_status need4(const void* p, const char* name) {
  if (!p) return fail(LIK_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned4(p)) return fail(LIK_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return LIK_OK;
}
lik_status need16(const void* p, const char* name) {
  if (!p) return fail(LIK_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(LIK_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return LIK_OK;
}

int64_t size_of(lik_dtype t) { return t == LIK_F32 ? 4 : (t == LIK_F16 || t == LIK_BF16 ? 2 : 0); }

bool valid_block(int64_t bs) { return bs >= 16 && bs <= 256 && (bs & (bs - 1)) == 0; }
bool valid_dim(int64_t dim) { return dim == 64 || dim == 128 || dim == 256; }

#define LIK_TRY(x)                     \
  do {                                 \
    const lik_status st_ = (x);        \
    if (st_ != LIK_OK) return st_;     \
  } while (0)

lik_status check_blocks(int64_t num_blocks, int64_t block_size) {
  if (num_blocks < 0)
    return fail(LIK_ERR_INVALID_ARG, "negative size (num_blocks %lld)", (long long)num_blocks);
  if (!valid_block(block_size))
    return fail(LIK_ERR_INVALID_ARG, "block_size must be a power of two from 16 to 256 (got %lld)",
                (long long)block_size);
  if (num_blocks > INT32_MAX / block_size)
    return fail(LIK_ERR_UNSUPPORTED, "num_blocks x block_size must be below 2^31");
  return LIK_OK;
}

lik_status check_table(int64_t S, int64_t max_blocks, int64_t table_ld, int64_t block_size) {
  if (S < 0 || max_blocks < 0)
    return fail(LIK_ERR_INVALID_ARG, "negative size (S %lld, max_blocks %lld)", (long long)S,
                (long long)max_blocks);
  if (table_ld < max_blocks)
    return fail(LIK_ERR_INVALID_ARG, "row stride table_ld %lld is less than max_blocks %lld",
                (long long)table_ld, (long long)max_blocks);
  if (mul_ok({S, table_ld, 4}) < 0) return fail(LIK_ERR_INVALID_ARG, "S x row stride overflows");
  if (S > lik::kCacheMaxSeqs)
    return fail(LIK_ERR_UNSUPPORTED, "S must be at most 2^20 (got %lld)", (long long)S);
  if (max_blocks > INT32_MAX / block_size)
    return fail(LIK_ERR_UNSUPPORTED, "max_blocks x block_size must be below 2^31");
  return LIK_OK;
}

// Sizes and pointers of a cache that is there (num_blocks > 0).
lik_status check_cache(const void* k, const void* v, const float* ks, const float* vs, int64_t n,
                       int64_t heads, int64_t block_size, int64_t dim, int64_t k_stride,
                       int64_t v_stride) {
  const int64_t least = heads * block_size * dim;
  if (k_stride < least || v_stride < least)
    return fail(LIK_ERR_INVALID_ARG,
                "block strides %lld, %lld are less than a block's %lld bytes", (long long)k_stride,
                (long long)v_stride, (long long)least);
  if (k_stride % 16 || v_stride % 16)
    return fail(LIK_ERR_INVALID_ARG, "block strides must be multiples of 16");
  if (mul_ok({n, k_stride}) < 0 || mul_ok({n, v_stride}) < 0 || mul_ok({n, heads, 4}) < 0)
    return fail(LIK_ERR_INVALID_ARG, "num_blocks x block stride overflows");
  if (n == 0) return LIK_OK;
  LIK_TRY(need16(k, "k_cache"));
  LIK_TRY(need16(v, "v_cache"));
  LIK_TRY(need4(ks, "k_scale"));
  LIK_TRY(need4(vs, "v_scale"));
  return LIK_OK;
}

// Rows [T][heads][dim] with a token stride of ld elements, 16-byte aligned.
lik_status check_tokens(const void* p, const char* name, int64_t T, int64_t width, int64_t ld,
                        int64_t size) {
  if (ld < width)
    return fail(LIK_ERR_INVALID_ARG, "token stride of %s, %lld, is less than %lld", name,
                (long long)ld, (long long)width);
  if (ld * size % 16)
    return fail(LIK_ERR_INVALID_ARG, "token stride of %s must be a multiple of 16 bytes", name);
  if (mul_ok({T, ld, size}) < 0)
    return fail(LIK_ERR_INVALID_ARG, "T x token stride of %s overflows", name);
  return need16(p, name);
}

lik_status check_heads(int64_t kv_heads, int64_t dim) {
  if (kv_heads <= 0)
    return fail(LIK_ERR_INVALID_ARG, "kv_heads must be positive (got %lld)", (long long)kv_heads);
  if (kv_heads > 65535)
    return fail(LIK_ERR_UNSUPPORTED, "kv_heads must be below 2^16 (got %lld)", (long long)kv_heads);
  if (!valid_dim(dim))
    return fail(LIK_ERR_UNSUPPORTED, "dim must be 64, 128 or 256 (got %lld)", (long long)dim);
  return LIK_OK;
}

// Whether blocks of one array alternate with the other's without touching them.
bool interleaved(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int64_t bytes) {
  if (k_stride != v_stride) return false;
  const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(v) - reinterpret_cast<uintptr_t>(k));
  const int64_t d = ((apart % k_stride) + k_stride) % k_stride;
  return d >= bytes && k_stride - d >= bytes;
}

lik_status launched(hipError_t e) {
  if (e != hipSuccess) return fail(LIK_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
  return ok();
}

// The sizes of an attention call that its workspace depends on.
lik_status check_attend(int64_t T, int64_t S, int64_t q_heads, int64_t kv_heads, int64_t dim,
                        lik_dtype dtype) {
  if (!size_of(dtype)) return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d for q", (int)dtype);
  if (T < 0 || S < 0)
    return fail(LIK_ERR_INVALID_ARG, "negative size (T %lld, S %lld)", (long long)T, (long long)S);
  LIK_TRY(check_heads(kv_heads, dim));
  if (q_heads <= 0 || q_heads % kv_heads)
    return fail(LIK_ERR_INVALID_ARG, "q_heads %lld is no multiple of kv_heads %lld",
                (long long)q_heads, (long long)kv_heads);
  if (T > INT32_MAX / q_heads)
    return fail(LIK_ERR_UNSUPPORTED, "T x q_heads must be below 2^31 (got %lld x %lld)",
                (long long)T, (long long)q_heads);
  if (S > lik::kCacheMaxSeqs)
    return fail(LIK_ERR_UNSUPPORTED, "S must be at most 2^20 (got %lld)", (long long)S);
  return LIK_OK;
}

}  // namespace

extern "C" {

lik_status lik_cache_tables(const int32_t* old_len, const int32_t* new_len, int64_t S,
                            int64_t block_size, int32_t* block_table, int64_t max_blocks,
                            int64_t table_ld, int32_t* ring, int64_t num_blocks,
                            int32_t* ring_state, int32_t* granted, int32_t* token_offsets,
                            int32_t* slots, int64_t T, void* stream) {
  LIK_TRY(check_blocks(num_blocks, block_size));
  LIK_TRY(check_table(S, max_blocks, table_ld, block_size));
  if (T < 0) return fail(LIK_ERR_INVALID_ARG, "negative size (T %lld)", (long long)T);
  if (T > INT32_MAX) return fail(LIK_ERR_UNSUPPORTED, "T must be below 2^31");
  if (S > 0) {
    LIK_TRY(need4(old_len, "old_len"));
    LIK_TRY(need4(new_len, "new_len"));
    LIK_TRY(need4(granted, "granted"));
    if (max_blocks > 0) LIK_TRY(need4(block_table, "block_table"));
  }
  if (num_blocks > 0) LIK_TRY(need4(ring, "ring"));
  LIK_TRY(need4(ring_state, "ring_state"));
  LIK_TRY(need4(token_offsets, "token_offsets"));
  if (T > 0) LIK_TRY(need4(slots, "slots"));
  const int64_t table = S > 0 ? ((S - 1) * table_ld + max_blocks) * 4 : 0;
  const Span in[] = {{old_len, S * 4}, {new_len, S * 4}};
  const Span out[] = {{block_table, table}, {ring, num_blocks * 4}, {ring_state, 16},
                      {granted, S * 4},     {token_offsets, (S + 1) * 4}, {slots, T * 4}};
  if (lik::any_overlap(in, out))
    return fail(LIK_ERR_INVALID_ARG, "an output overlaps an input or another output");
  LIK_TRY(check_device());
  const lik::TablesArgs a{old_len, new_len, (int)S, (int)block_size, block_table, (int)max_blocks,
                          table_ld, ring, (int)num_blocks, ring_state, granted, token_offsets,
                          slots, (int)T};
  return launched(lik::run_tables(a, static_cast<hipStream_t>(stream)));
}

lik_status lik_cache_append(const void* k, const void* v, lik_dtype dtype, int64_t T, int64_t k_ld,
                            int64_t v_ld, const int32_t* slots, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, int64_t num_blocks, int64_t kv_heads,
                            int64_t block_size, int64_t dim, int64_t k_stride, int64_t v_stride,
                            void* stream) {
  const int64_t size = size_of(dtype);
  if (!size) return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d for k and v", (int)dtype);
  if (T < 0) return fail(LIK_ERR_INVALID_ARG, "negative size (T %lld)", (long long)T);
  LIK_TRY(check_blocks(num_blocks, block_size));
  LIK_TRY(check_heads(kv_heads, dim));
  LIK_TRY(check_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, kv_heads, block_size, dim,
                      k_stride, v_stride));
  if (T == 0 || num_blocks == 0) return ok();
  // the kernel looks 127 tokens beyond the one that a run begins with
  if (T >= INT32_MAX - 255)
    return fail(LIK_ERR_UNSUPPORTED, "T must be below 2^31 - 2^8 (got %lld)", (long long)T);
  const int64_t width = kv_heads * dim;
  LIK_TRY(check_tokens(k, "k", T, width, k_ld, size));
  LIK_TRY(check_tokens(v, "v", T, width, v_ld, size));
  LIK_TRY(need4(slots, "slots"));
  // a block's bytes interleave with the other cache's where both lie in one array
  const Span in[] = {{k, ((T - 1) * k_ld + width) * size}, {v, ((T - 1) * v_ld + width) * size},
                     {slots, T * 4}};
  const Span caches[] = {{k_cache, (num_blocks - 1) * k_stride + width * block_size}};
  const Span more[] = {{v_cache, (num_blocks - 1) * v_stride + width * block_size}};
  const Span scales[] = {{k_scale, num_blocks * kv_heads * 4}, {v_scale, num_blocks * kv_heads * 4}};
  if (lik::any_overlap(in, caches) || lik::any_overlap(in, more) || lik::any_overlap(in, scales) ||
      lik::any_overlap(caches, scales) || lik::any_overlap(more, scales))
    return fail(LIK_ERR_INVALID_ARG, "an output overlaps an input or another output");
  if (lik::overlap(caches[0], more[0]) && !interleaved(k_cache, v_cache, k_stride, v_stride,
                                                       width * block_size))
    return fail(LIK_ERR_INVALID_ARG, "k_cache overlaps v_cache");
  LIK_TRY(check_device());
  const lik::AppendArgs a{{k, v}, {k_ld, v_ld}, dtype, (int)T, (int)kv_heads, (int)dim,
                          (int)block_size, (int)num_blocks, slots,
                          {{static_cast<uint8_t*>(k_cache), k_scale, k_stride},
                           {static_cast<uint8_t*>(v_cache), v_scale, v_stride}}};
  return launched(lik::run_append(a, static_cast<hipStream_t>(stream)));
}

size_t lik_cache_workspace_bytes(int64_t T, int64_t S, int64_t q_heads, int64_t kv_heads,
                                 int64_t dim, lik_dtype dtype) {
  if (check_attend(T, S, q_heads, kv_heads, dim, dtype) != LIK_OK) return SIZE_MAX;
  ok();
  return T == 0 ? 0 : lik::attend_workspace(T, S, q_heads, kv_heads, dim, dtype);
}

lik_status lik_cache_attention(const void* q, lik_dtype dtype, int64_t T, int64_t q_heads,
                               int64_t q_ld, const int32_t* q_offsets, const int32_t* kv_len,
                               int64_t S, const int32_t* block_table, int64_t max_blocks,
                               int64_t table_ld, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, int64_t num_blocks,
                               int64_t kv_heads, int64_t block_size, int64_t dim, int64_t k_stride,
                               int64_t v_stride, float scale, void* out, int64_t out_ld, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  LIK_TRY(check_attend(T, S, q_heads, kv_heads, dim, dtype));
  LIK_TRY(check_blocks(num_blocks, block_size));
  LIK_TRY(check_table(S, max_blocks, table_ld, block_size));
  LIK_TRY(check_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, kv_heads, block_size, dim,
                      k_stride, v_stride));
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f))
    return fail(LIK_ERR_INVALID_ARG, "scale must be within [2^-64, 2^64]");
  if (T == 0) return ok();
  const int64_t size = size_of(dtype), width = q_heads * dim;
  LIK_TRY(check_tokens(q, "q", T, width, q_ld, size));
  LIK_TRY(check_tokens(out, "out", T, width, out_ld, size));
  if (S > 0) {
    LIK_TRY(need4(q_offsets, "q_offsets"));
    LIK_TRY(need4(kv_len, "kv_len"));
    if (max_blocks > 0) LIK_TRY(need4(block_table, "block_table"));
  }
  if (!aligned4(lse)) return fail(LIK_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const int64_t cache = kv_heads * block_size * dim;
  const Span in[] = {{q, ((T - 1) * q_ld + width) * size},
                     {q_offsets, (S + 1) * 4},
                     {kv_len, S * 4},
                     {block_table, S > 0 ? ((S - 1) * table_ld + max_blocks) * 4 : 0},
                     {k_cache, num_blocks > 0 ? (num_blocks - 1) * k_stride + cache : 0},
                     {v_cache, num_blocks > 0 ? (num_blocks - 1) * v_stride + cache : 0},
                     {k_scale, num_blocks * kv_heads * 4},
                     {v_scale, num_blocks * kv_heads * 4}};
  const Span outs[] = {{out, ((T - 1) * out_ld + width) * size}, {lse, lse ? T * q_heads * 4 : 0}};
  if (lik::any_overlap(in, outs))
    return fail(LIK_ERR_INVALID_ARG, "an output overlaps an input or another output");
  const size_t need = lik::attend_workspace(T, S, q_heads, kv_heads, dim, dtype);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(LIK_ERR_INVALID_ARG, "workspace too small: %zu bytes needed, %zu given", need,
                  workspace ? workspace_bytes : (size_t)0);
    if (!aligned16(workspace))
      return fail(LIK_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  }
  LIK_TRY(check_device());
  const lik::AttendArgs a{q, dtype, (int)T, (int)q_heads, (int)kv_heads, (int)dim, (int)S, q_ld,
                          q_offsets, kv_len, block_table, (int)max_blocks, table_ld,
                          {static_cast<uint8_t*>(const_cast<void*>(k_cache)),
                           const_cast<float*>(k_scale), k_stride},
                          {static_cast<uint8_t*>(const_cast<void*>(v_cache)),
                           const_cast<float*>(v_scale), v_stride},
                          (int)num_blocks, (int)block_size, scale, out, out_ld, lse};
  return launched(
      lik::run_attend(a, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"

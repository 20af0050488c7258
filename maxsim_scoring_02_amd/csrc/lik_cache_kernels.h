// Internal interface between the C ABI of the 8-bit cache and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lik.h"
#include "lik_cache.h"

namespace lik {

constexpr int64_t kCacheMaxSeqs = int64_t(1) << 20;

struct TablesArgs {
  const int32_t* old_len;
  const int32_t* new_len;
  int S, block_size;
  int32_t* table;
  int max_blocks;
  int64_t table_ld;
  int32_t* ring;
  int num_blocks;
  int32_t* state;
  int32_t* granted;
  int32_t* offsets;
  int32_t* slots;
  int T;
};

// Blocks of one of the two caches, and their scales.
struct CachePart {
  uint8_t* codes;
  float* scale;
  int64_t stride;                        // bytes from block to block
};

struct AppendArgs {
  const void* x[2];                      // k, v
  int64_t ld[2];
  lik_dtype dtype;
  int T, heads, dim, block_size, num_blocks;
  const int32_t* slots;
  CachePart part[2];
};

struct AttendArgs {
  const void* q;
  lik_dtype dtype;
  int T, q_heads, kv_heads, dim, S;
  int64_t q_ld;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  const int32_t* table;
  int max_blocks;
  int64_t table_ld;
  CachePart k, v;
  int num_blocks, block_size;
  float scale;
  void* out;
  int64_t out_ld;
  float* lse;
};

hipError_t run_tables(const TablesArgs& a, hipStream_t s);
hipError_t run_append(const AppendArgs& a, hipStream_t s);
size_t attend_workspace(int64_t T, int64_t S, int64_t q_heads, int64_t kv_heads, int64_t dim,
                        lik_dtype dtype);
hipError_t run_attend(const AttendArgs& a, char* ws, hipStream_t s);

}  // namespace lik

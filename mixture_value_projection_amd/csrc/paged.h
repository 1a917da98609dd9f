// Launch interface of the paged key-value cache's kernels, between the C ABI
// (paged_api.hip) and the kernels, and the helpers that they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace mova {

// Requests one call takes (paged_plan.hip keeps four numbers of each in LDS).
constexpr int kMaxRequests = 2048;

// Element type of a cache pool (mova_cache_dtype of include/mova.h).
enum CacheDtype { kCacheBf16 = 0, kCacheFp8 = 1 };

struct PlanArgs {
  const int32_t* cached;  // [B]
  const int32_t* fresh;   // [B], < 0: the request has ended
  int B, T, block_size, max_blocks;
  int32_t* table;        // [B, max_blocks]
  int32_t* free_blocks;  // [free_capacity], a stack
  int free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* seq_lens;  // [B]
  int32_t* cu_new;    // [B + 1]
  int64_t* slots;     // [T]
  int32_t* positions; // [T]
};
hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream);

struct StoreArgs {
  const __bf16* k;  // [T, H, D] or null
  const __bf16* v;  // [T, H, D] or null
  int T, H, D;
  void* k_cache;
  void* v_cache;
  int dtype;
  const float* k_scale;  // [H] or null (1)
  const float* v_scale;
  long long num_slots;
  int block_size;
  const int64_t* slots;  // [T]
  __bf16* bounds;        // [num_blocks, H, 2, D] or null
};
hipError_t launch_kv_store(const StoreArgs& a, hipStream_t stream);

struct SelectArgs {
  const __bf16* q;       // [B, Hq, D]
  const __bf16* bounds;  // [num_blocks, H, 2, D]
  int num_blocks, block_size;
  const int32_t* table;  // [B, max_blocks]
  int max_blocks;
  const int32_t* seq_lens;  // [B]
  int B, Hq, H, D;
  int keep, first, last;
  int32_t* sel;    // [B, H, keep]
  double* scores;  // [B, H, max_blocks] scratch
};
hipError_t launch_block_select(const SelectArgs& a, hipStream_t stream);

struct AttentionArgs {
  const __bf16* q;  // [B, Hq, D]
  const void* k_cache;
  const void* v_cache;
  int dtype;
  const float* k_scale;  // [H] or null
  const float* v_scale;
  int num_blocks, block_size;
  const int32_t* table;  // [B, max_blocks]
  int max_blocks;
  const int32_t* seq_lens;  // [B]
  const int32_t* sel;       // [B, H, keep] or null
  int keep;
  int B, Hq, H, D;
  float scale;
  int window;  // 0: none
  __bf16* out;  // [B, Hq, D]
  float* lse;   // [B, Hq] or null
  float* part;  // scratch of attention_scratch_floats
};
// Floats of scratch; depends on the sizes alone.
size_t attention_scratch_floats(int B, int Hq, int H, int D, int max_blocks, int block_size,
                                int keep);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream);

// ---- device helpers ---------------------------------------------------------

// Tokens of request b: its length, kept inside its row of the block table.
__device__ __forceinline__ int request_len(const int32_t* seq_lens, int b, int max_blocks,
                                           int block_size) {
  return min(max(seq_lens[b], 0), max_blocks * block_size);
}

}  // namespace mova

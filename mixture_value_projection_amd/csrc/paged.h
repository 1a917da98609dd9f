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
  unsigned long long* scratch;  // [B, H, max_blocks]
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

// n / d for 0 <= n < 2^31 as a product and a shift (d > 0).  With
// s = ceil(log2 d), mul = floor(2^(31 + s) / d) + 1 exceeds 2^(31 + s) / d by at
// most 1, so the product exceeds n / d by less than n / 2^(31 + s) < 1 / d.
struct FastDiv {
  uint32_t mul, shift;
};
inline FastDiv make_fast_div(int d) {
  uint32_t s = 0;
  while ((1ll << s) < d) ++s;
  return {(uint32_t)((1ull << (31 + s)) / (unsigned)d + 1), 31 + s};
}
__device__ __forceinline__ int fast_div(int n, FastDiv f) {
  return (int)(((unsigned long long)(uint32_t)n * f.mul) >> f.shift);
}

// Exclusive scan of one number a thread over a workgroup of kWaves waves;
// *total gets the sum.  `tmp` holds one number a wave and may be used again
// after the next barrier.
template <int kWaves>
__device__ __forceinline__ long long block_exclusive_scan(long long x, long long* tmp,
                                                          long long* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long inc = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long up = __shfl_up(inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 63) tmp[wave] = inc;
  __syncthreads();
  long long before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += tmp[w];
    sum += tmp[w];
  }
  *total = sum;
  return before + inc - x;
}

// A line of work over a ragged batch: request b brings cost(b) units, one
// request after the other, and each of gridDim.x workgroups takes an equal
// stretch [start, end) of them.  The workgroup finds the request that its
// stretch begins in, and that request's first unit, from the lengths alone.
struct Line {
  long long stretch, start, end;
  long long first;  // first unit of request b
  int b;
};
struct LineShared {
  long long tmp[4], first;
  int b;
};
// For workgroups of 256 threads.  False: nothing to do.  `prefix` (null, or
// B + 1 numbers): workgroup 0 writes the requests' first units and the stretch.
template <class Cost>
__device__ __forceinline__ bool line_begin(int B, Cost cost, LineShared& sh, long long* prefix,
                                           Line* line) {
  const int per = ceil_div(B, 256);
  const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += cost(b);
  long long before = block_exclusive_scan<4>(mine, sh.tmp, &total);
  line->stretch = max((total + gridDim.x - 1) / gridDim.x, 1ll);
  line->start = line->stretch * blockIdx.x;
  line->end = min(line->start + line->stretch, total);
  if (before <= line->start && line->start < before + mine) {
    long long at = before;
    int b = b0;
    for (long long c; line->start >= at + (c = cost(b)); ++b) at += c;
    sh.b = b;
    sh.first = at;
  }
  if (prefix != nullptr && blockIdx.x == 0) {
    for (int b = b0; b < b1; ++b) {
      prefix[b] = before;
      before += cost(b);
    }
    if (threadIdx.x == 0) prefix[B] = line->stretch;
  }
  if (line->start >= total) return false;
  __syncthreads();
  line->b = sh.b;
  line->first = sh.first;
  return true;
}

// Tokens of request b: its length, kept inside its row of the block table.
__device__ __forceinline__ int request_len(const int32_t* seq_lens, int b, int max_blocks,
                                           int block_size) {
  return min(max(seq_lens[b], 0), max_blocks * block_size);
}

}  // namespace mova

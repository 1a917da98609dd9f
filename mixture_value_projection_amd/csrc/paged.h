// Launch interface of the paged key-value cache's kernels, between the C ABI
// (paged_api.hip) and the kernels, and the helpers that they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
  unsigned long long* scratch;  // select_scratch_words
};
// Scratch, in 8-byte words: a word a block, in rows that hold whole tiles of
// kSelectTile blocks (the choice reads whole tiles); then a word a tile.
constexpr int kSelectTile = 16;
__host__ __device__ constexpr size_t select_stride(int max_blocks) {
  return ((size_t)max_blocks + kSelectTile - 1) / kSelectTile * kSelectTile;
}
__host__ __device__ constexpr size_t select_tiles_at(int B, int H, int max_blocks) {
  return (size_t)B * H * select_stride(max_blocks);
}
inline size_t select_scratch_words(int B, int H, int max_blocks) {
  return select_tiles_at(B, H, max_blocks) +
         (size_t)B * H * (select_stride(max_blocks) / kSelectTile);
}
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
size_t attention_scratch_floats(int B, int Hq, int H, int D);
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

// ---- sums over a wave in registers (no LDS round trips) ----

// x of the lane that the DPP control names; 0 where there is none or the row
// is masked out.
template <int kCtrl, int kRows = 0xf>
__device__ __forceinline__ int dpp_or_0(int x) {
  return __builtin_amdgcn_update_dpp(0, x, kCtrl, kRows, 0xf, true);
}
template <int kCtrl, int kRows = 0xf>
__device__ __forceinline__ double dpp_or_0(double x) {
  int2 u = __builtin_bit_cast(int2, x);
  u.x = dpp_or_0<kCtrl, kRows>(u.x);
  u.y = dpp_or_0<kCtrl, kRows>(u.y);
  return __builtin_bit_cast(double, u);
}
// Inclusive sum over lanes 0 .. lane (int or double).
template <class X>
__device__ __forceinline__ X wave_scan(X x) {
  x += dpp_or_0<0x111>(x);       // row_shr 1, 2, 4, 8
  x += dpp_or_0<0x112>(x);
  x += dpp_or_0<0x114>(x);
  x += dpp_or_0<0x118>(x);
  x += dpp_or_0<0x142, 0xa>(x);  // row_bcast 15, 31
  x += dpp_or_0<0x143, 0xc>(x);
  return x;
}
__device__ __forceinline__ float wave_sum(float x) {
  auto step = [&](int moved) { x += __builtin_bit_cast(float, moved); };
  step(dpp_or_0<0x111>(__builtin_bit_cast(int, x)));
  step(dpp_or_0<0x112>(__builtin_bit_cast(int, x)));
  step(dpp_or_0<0x114>(__builtin_bit_cast(int, x)));
  step(dpp_or_0<0x118>(__builtin_bit_cast(int, x)));
  step(dpp_or_0<0x142, 0xa>(__builtin_bit_cast(int, x)));
  step(dpp_or_0<0x143, 0xc>(__builtin_bit_cast(int, x)));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ int read_lane(int x, int lane) {
  return __builtin_amdgcn_readlane(x, lane);
}
__device__ __forceinline__ double read_lane(double x, int lane) {
  int2 u = __builtin_bit_cast(int2, x);
  u.x = __builtin_amdgcn_readlane(u.x, lane);
  u.y = __builtin_amdgcn_readlane(u.y, lane);
  return __builtin_bit_cast(double, u);
}
// op over the wave of 32-bit x, in all lanes.
template <class X, class Op>
__device__ __forceinline__ X wave_reduce(X x, Op op) {
  auto step = [&](auto ctrl, auto rows) {
    const int i = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(
        X, __builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
  };
  using std::integral_constant;
  x = op(x, step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{}));
  x = op(x, step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{}));
  x = op(x, step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{}));
  x = op(x, step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{}));
  x = op(x, step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{}));
  x = op(x, step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{}));
  return __builtin_bit_cast(X, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// Exclusive scan of one number a thread over a workgroup of kWaves waves;
// *total gets the sum (below 2^53).  `tmp` holds one number a wave and may be
// used again after the next barrier.
template <int kWaves>
__device__ __forceinline__ long long block_exclusive_scan(long long x, long long* tmp,
                                                          long long* total) {
  const int wave = threadIdx.x >> 6;
  const long long inc = (long long)wave_scan((double)x);
  if ((threadIdx.x & 63) == 63) tmp[wave] = inc;
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

// floor(x / y) for 0 <= x < 2^52 and 0 < y < 2^52: the quotient is at least
// 1 / y > 2^-52 x / y away from the next whole number, so rounding it cannot
// reach that.
__device__ __forceinline__ long long floor_div(long long x, long long y) {
  return (long long)((double)x / (double)y);
}

// A line of work over a ragged batch: request b brings cost(b) units, one
// request after the other, and each of gridDim.x workgroups takes an equal
// stretch [start, end) of them (2^52 units at most).  The workgroup finds the
// request that its stretch begins in, and that request's first unit, from the
// lengths alone.
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
// Up to 64 requests each wave adds up the line for itself, one request a lane;
// above, the workgroup does.
template <class Cost>
__device__ __forceinline__ bool line_begin(int B, Cost cost, LineShared& sh, long long* prefix,
                                           Line* line) {
  if (B <= 64) {
    const int lane = threadIdx.x & 63;
    const double mine = lane < B ? (double)cost(lane) : 0.0;
    const double upto = wave_scan(mine), before = upto - mine;
    const long long total = (long long)read_lane(upto, 63);
    line->stretch = max(floor_div(total + gridDim.x - 1, gridDim.x), 1ll);
    line->start = line->stretch * blockIdx.x;
    line->end = min(line->start + line->stretch, total);
    if (prefix != nullptr && blockIdx.x == 0 && threadIdx.x < 64) {
      if (lane < B) prefix[lane] = (long long)before;
      if (lane == 0) prefix[B] = line->stretch;
    }
    if (line->start >= total) return false;
    const double at = (double)line->start;
    line->b = __ffsll((unsigned long long)__ballot(before <= at && at < upto)) - 1;
    line->first = (long long)read_lane(before, line->b);
    return true;
  }
  const int per = ceil_div(B, 256);
  const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += cost(b);
  long long before = block_exclusive_scan<4>(mine, sh.tmp, &total);
  line->stretch = max(floor_div(total + gridDim.x - 1, gridDim.x), 1ll);
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
  line->b = __builtin_amdgcn_readfirstlane(sh.b);
  line->first = (long long)read_lane((double)sh.first, 0);
  return true;
}

// Tokens of request b: its length, kept inside its row of the block table.
__device__ __forceinline__ int request_len(const int32_t* seq_lens, int b, int max_blocks,
                                           int block_size) {
  return min(max(seq_lens[b], 0), max_blocks * block_size);
}

// Direct-to-LDS loads of 16 (kStream: with the non-temporal hint) and 4 bytes a
// lane, to consecutive places.
template <bool kStream>
__device__ __forceinline__ void piece_to_lds(const void* from, void* to) {
  if constexpr (kStream)
    __builtin_amdgcn_global_load_lds(from, (lds_void*)to, 16, 0, kLdsLoadNonTemporal);
  else
    __builtin_amdgcn_global_load_lds(from, (lds_void*)to, 16, 0, 0);
}
__device__ __forceinline__ void word_to_lds(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds(from, (lds_void*)to, 4, 0, 0);
}

// A use of x: the load behind it is waited for here and not later.
template <class X>
__device__ __forceinline__ void loaded(X& x) {
  asm volatile("" : "+v"(x));
}

// Waits until at most `left` <= kMost groups of kOps vector-memory operations
// are outstanding, and for LDS.
template <int kMost, int kOps>
__device__ __forceinline__ void wait_groups(int left) {
  if constexpr (kMost == 0) {
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));
  } else {
    if (left == kMost) __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(kMost * kOps));
    else wait_groups<kMost - 1, kOps>(left);
  }
}

}  // namespace mova

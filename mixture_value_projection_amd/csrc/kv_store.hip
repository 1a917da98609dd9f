// Keys and values of a step's tokens stored into the paged pools, and the key
// bounds of the blocks they touch.
//
// Copying: a wave takes one token row and 64 pieces of 8 channels of it.
//
// Bounds: the last row of a run (the tokens that went to consecutive rows of
// one block) stands for the run's block.  A workgroup looks for such rows among
// a few tokens and forms their blocks' bounds, over the run's rows as they came
// and the block's rows before them, a quarter of the rows a wave, eight asked
// for at a time.  No wave reads what another writes, so the bounds go along
// with the copying in one launch, and their workgroups come first, being the
// longer way: 8192 rows of keys and values to 8 bits take 14 us without bounds
// and 16 us with them (22 us with the bounds formed by the wave that copies the
// run's last row).  Rounding to 8 bits keeps the order, so only the smallest
// and largest of a run's rows are rounded for them.
#include <algorithm>

#include "paged.h"

namespace mova {

namespace {

constexpr float kFp8Max = 448.f;
constexpr int kRowsAtOnce = 8;

// Beyond +-448 is +-448, NaN stays.
__device__ __forceinline__ float fp8_clamp(float x) {
  x = x > kFp8Max ? kFp8Max : x;
  return x < -kFp8Max ? -kFp8Max : x;
}

// e4m3 of 8 elements, nearest even.
__device__ __forceinline__ uint2 fp8_pack(const Frag16& x, float scale) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = fp8_clamp((float)x.h[i] / scale);
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], b, true);
  return uint2{(uint32_t)a, (uint32_t)b};
}

// 8 elements as the pool holds them.
template <bool kFp8>
struct Stored {
  Frag16 x;  // bf16
  __device__ __forceinline__ void take(const Frag16& v, float) { x = v; }
  __device__ __forceinline__ void load(const void* p, size_t at) { x.u = load16((const bf16_t*)p + at); }
  __device__ __forceinline__ void store(void* p, size_t at) const { store16((bf16_t*)p + at, x.u); }
  __device__ __forceinline__ float get(int i) const { return (float)x.h[i]; }
};
template <>
struct Stored<true> {
  uint2 w;
  __device__ __forceinline__ void take(const Frag16& v, float scale) { w = fp8_pack(v, scale); }
  __device__ __forceinline__ void load(const void* p, size_t at) {
    w = *reinterpret_cast<const uint2*>((const uint8_t*)p + at);
  }
  __device__ __forceinline__ void store(void* p, size_t at) const {
    *reinterpret_cast<uint2*>((uint8_t*)p + at) = w;
  }
  __device__ __forceinline__ float get(int i) const {
    return __builtin_amdgcn_cvt_f32_fp8((int)((i < 4 ? w.x : w.y) >> (8 * (i & 3))), 0);
  }
};

}  // namespace

// Workgroups [0, bounds_groups) form bounds, of `tokens` tokens each and one
// piece group; the others copy.
template <bool kFp8>
__global__ __launch_bounds__(256, 6) void kv_store_kernel(StoreArgs a, int bounds_groups, int tokens) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = a.H * a.D;
  const int groups = ceil_div(width, 512);
  if ((int)blockIdx.x >= bounds_groups) {
    const int items = a.T * groups;  // at most 2^29
    const int step = ((int)gridDim.x - bounds_groups) * 4;
    for (int item = ((int)blockIdx.x - bounds_groups) * 4 + wave; item < items; item += step) {
      const int t = item / groups;
      const int c = ((item - t * groups) * 64 + lane) * 8;
      const long long s = a.slots[t];
      if (s < 0 || s >= a.num_slots || c >= width) continue;
      const int head = c / a.D;
      const size_t from = (size_t)t * width + c, to = (size_t)s * width + c;
      Frag16 x, y;
      if (a.k != nullptr) x.u = load16(a.k + from);
      if (a.v != nullptr) y.u = load16(a.v + from);
      Stored<kFp8> e;
      if (a.k != nullptr) {
        e.take(x, a.k_scale == nullptr ? 1.f : a.k_scale[head]);
        e.store(a.k_cache, to);
      }
      if (a.v != nullptr) {
        e.take(y, a.v_scale == nullptr ? 1.f : a.v_scale[head]);
        e.store(a.v_cache, to);
      }
    }
    return;
  }

  __shared__ __attribute__((aligned(16))) float parts[3][64][16];
  const int group = blockIdx.x % groups;
  const int c = (group * 64 + lane) * 8;
  const bool live = c < width;
  const int head = live ? c / a.D : 0;
  // A lane a token: which are the last of a run.
  const int first = (int)(blockIdx.x / groups) * tokens;
  bool ends = false;
  if (lane < tokens && first + lane < a.T) {
    const int t = first + lane;
    const long long s = a.slots[t], next = a.slots[min(t + 1, a.T - 1)];
    const bool goes_on = t + 1 < a.T && next == s + 1 && (s + 1) % a.block_size != 0;
    ends = s >= 0 && s < a.num_slots && !goes_on;
  }
  for (uint64_t found = __ballot(ends); found != 0; found &= found - 1) {
    const int t = first + __ffsll((unsigned long long)found) - 1;
    const long long s = a.slots[t];
    const long long page = s / a.block_size;
    const int off = (int)(s - page * a.block_size);
    // Rows of the run before this one: a lane a row.
    int before = 0;
    for (const int most = min(off, t); before < most;) {
      const int i = before + 1 + lane;
      const uint64_t m = ~__ballot(i <= most && a.slots[t - i] == s - i);
      if (m != 0) {
        before += __ffsll((unsigned long long)m) - 1;
        break;
      }
      before += 64;
    }
    // A NaN key makes its channel's bounds NaN.
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo[j] = __builtin_huge_valf();
      hi[j] = -__builtin_huge_valf();
    }
    auto meet = [&](int j, float f, float g) {
      lo[j] = __builtin_elementwise_minimum(lo[j], f);
      hi[j] = __builtin_elementwise_maximum(hi[j], g);
    };
    // This wave's rows, counted upwards from the last.
    const int per = ceil_div(off + 1, 4);
    const int i0 = wave * per, i1 = min(i0 + per, off + 1);
    const int fresh = min(i1, before + 1);  // [i0, fresh) are the run's
    if (live) {
#pragma unroll 1
      for (int i = i0; i < fresh; i += kRowsAtOnce) {
        Frag16 x[kRowsAtOnce];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
          x[r].u = load16(a.k + (size_t)(t - min(i + r, fresh - 1)) * width + c);
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j) meet(j, (float)x[r].h[j], (float)x[r].h[j]);
      }
      if (kFp8 && i0 < fresh) {
        const float scale = a.k_scale == nullptr ? 1.f : a.k_scale[head];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int w = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_clamp(lo[j] / scale),
                                                        fp8_clamp(hi[j] / scale), 0, false);
          lo[j] = __builtin_amdgcn_cvt_f32_fp8(w, 0);
          hi[j] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
        }
      }
#pragma unroll 1
      for (int i = max(i0, fresh); i < i1; i += kRowsAtOnce) {
        Stored<kFp8> v[kRowsAtOnce];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
          v[r].load(a.k_cache, (size_t)(s - min(i + r, i1 - 1)) * width + c);
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j) meet(j, v[r].get(j), v[r].get(j));
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        parts[wave - 1][lane][j] = lo[j];
        parts[wave - 1][lane][8 + j] = hi[j];
      }
    }
    __syncthreads();
    if (wave == 0 && live) {
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) meet(j, parts[w][lane][j], parts[w][lane][8 + j]);
      bf16x8 l, h;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        l[j] = (bf16_t)lo[j];
        h[j] = (bf16_t)hi[j];
      }
      bf16_t* dst = a.bounds + ((size_t)page * a.H + head) * 2 * a.D + (c - head * a.D);
      *reinterpret_cast<bf16x8*>(dst) = l;
      *reinterpret_cast<bf16x8*>(dst + a.D) = h;
    }
    __syncthreads();
  }
}

hipError_t launch_kv_store(const StoreArgs& a, hipStream_t stream) {
  const int groups = ceil_div(a.H * a.D, 512);
  // A launch has fewer than 2^32 threads: of very large calls a wave copies
  // several pieces (at most 2^21 workgroups here, and 2^23 for the bounds).
  const int copy = std::min((int)(((long long)a.T * groups + 3) / 4), 1 << 21);
  // A workgroup a token while there are few, so that a decode step's blocks
  // are worked on at once; prompts have about one run in block_size tokens.
  const int tokens = std::min(std::max(1, ceil_div(a.T, 256)), 64);
  const int bounds = a.bounds == nullptr ? 0 : ceil_div(a.T, tokens) * groups;
  if (a.dtype == kCacheFp8)
    kv_store_kernel<true><<<copy + bounds, 256, 0, stream>>>(a, bounds, tokens);
  else
    kv_store_kernel<false><<<copy + bounds, 256, 0, stream>>>(a, bounds, tokens);
  return hipGetLastError();
}

}  // namespace mova

// Keys and values of a step's tokens stored into the paged pools, and the key
// bounds of the blocks they touch.
#include <algorithm>

#include "paged.h"

namespace mova {

namespace {

constexpr float kFp8Max = 448.f;

// e4m3 of x / scale, nearest even, values beyond +-448 to +-448, NaN to NaN.
__device__ __forceinline__ float fp8_clamp(float x) {
  x = x > kFp8Max ? kFp8Max : x;
  return x < -kFp8Max ? -kFp8Max : x;
}

__device__ __forceinline__ uint32_t fp8_pack4(const float* x) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_clamp(x[0]), fp8_clamp(x[1]), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_clamp(x[2]), fp8_clamp(x[3]), w, true);
  return (uint32_t)w;
}

}  // namespace

// Thread (t, c): 8 channels of row t.
template <bool kFp8>
__global__ __launch_bounds__(256) void kv_store_kernel(StoreArgs a) {
  const int chunks = a.H * a.D / 8;
  const long long total = (long long)a.T * chunks;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long t = i / chunks;
    const int c = (int)(i - t * chunks) * 8;
    const long long s = a.slots[t];
    if (s < 0 || s >= a.num_slots) continue;
    auto one = [&](const __bf16* src, void* pool, const float* scale) {
      if (src == nullptr) return;
      const size_t from = (size_t)t * a.H * a.D + c, to = (size_t)s * a.H * a.D + c;
      Frag16 x;
      x.u = load16(src + from);
      if constexpr (!kFp8) {
        store16((bf16_t*)pool + to, x.u);
      } else {
        const float sc = scale == nullptr ? 1.f : scale[c / a.D];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (float)x.h[j] / sc;
        *reinterpret_cast<uint2*>((uint8_t*)pool + to) = uint2{fp8_pack4(f), fp8_pack4(f + 4)};
      }
    };
    one(a.k, a.k_cache, a.k_scale);
    one(a.v, a.v_cache, a.v_scale);
  }
}

// Thread (t, c), t the last row of its block that the call stored: bounds of 8
// channels over the block's rows up to it.
template <bool kFp8>
__global__ __launch_bounds__(256) void key_bounds_kernel(StoreArgs a) {
  const int chunks = a.H * a.D / 8;
  const long long total = (long long)a.T * chunks;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long t = i / chunks;
    const int c = (int)(i - t * chunks) * 8;
    const long long s = a.slots[t];
    if (s < 0 || s >= a.num_slots) continue;
    const long long page = s / a.block_size;
    const int off = (int)(s - page * a.block_size);
    if (off + 1 < a.block_size && t + 1 < a.T && a.slots[t + 1] == s + 1) continue;
    float lo[8], hi[8];
    for (int r = 0; r <= off; ++r) {
      const size_t at = ((size_t)page * a.block_size + r) * a.H * a.D + c;
      float f[8];
      if constexpr (kFp8) {
        const uint2 w = *reinterpret_cast<const uint2*>((const uint8_t*)a.k_cache + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = __builtin_amdgcn_cvt_f32_fp8((int)(w.x >> (8 * j)), 0);
          f[4 + j] = __builtin_amdgcn_cvt_f32_fp8((int)(w.y >> (8 * j)), 0);
        }
      } else {
        Frag16 x;
        x.u = load16((const bf16_t*)a.k_cache + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (float)x.h[j];
      }
      // A NaN key makes its channel's bounds NaN.
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo[j] = (r == 0 || f[j] < lo[j] || f[j] != f[j]) ? f[j] : lo[j];
        hi[j] = (r == 0 || f[j] > hi[j] || f[j] != f[j]) ? f[j] : hi[j];
      }
    }
    bf16x8 l, h;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      l[j] = (bf16_t)lo[j];
      h[j] = (bf16_t)hi[j];
    }
    const int head = c / a.D, d = c - head * a.D;
    bf16_t* dst = a.bounds + ((size_t)page * a.H + head) * 2 * a.D + d;
    *reinterpret_cast<bf16x8*>(dst) = l;
    *reinterpret_cast<bf16x8*>(dst + a.D) = h;
  }
}

hipError_t launch_kv_store(const StoreArgs& a, hipStream_t stream) {
  const long long total = (long long)a.T * (a.H * a.D / 8);
  const int grid = (int)std::min<long long>((total + 255) / 256, 4096);
  if (a.dtype == kCacheFp8) kv_store_kernel<true><<<grid, 256, 0, stream>>>(a);
  else kv_store_kernel<false><<<grid, 256, 0, stream>>>(a);
  if (a.bounds != nullptr) {
    if (a.dtype == kCacheFp8) key_bounds_kernel<true><<<grid, 256, 0, stream>>>(a);
    else key_bounds_kernel<false><<<grid, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mova

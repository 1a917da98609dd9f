// Attention of a chunk of new tokens per request over the paged key-value cache
// that already holds them (prompts, chunks of prompts, drafts).
//
//   out_ti = sum_p exp(s_tip - m_ti) v_p / sum_p exp(s_tip - m_ti),  s_tip = scale q_ti . k_p
//
// over the positions p up to the token's own.
#include <algorithm>

#include "paged.h"

namespace mova {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Request b's rows of the packed tokens and positions in the cache.
struct Chunk {
  int row0, rows;  // packed rows [row0, row0 + rows)
  int at;          // position of the first
  int live;        // of the rows, how many have a token in the cache
};
__device__ __forceinline__ Chunk chunk_of(const ChunkArgs& a, int b) {
  const int most = a.max_blocks * a.block_size;
  Chunk c;
  c.row0 = min(max(a.cu_new[b], 0), a.T);
  c.rows = min(max(a.cu_new[b + 1], c.row0), a.T) - c.row0;
  c.at = min(max(a.cached[b], 0), most);
  const int len = a.num_blocks > 0 ? request_len(a.seq_lens, b, a.max_blocks, a.block_size) : 0;
  c.live = min(max(len - c.at, 0), c.rows);
  return c;
}

// 8 elements of the pool.
template <bool kFp8>
__device__ __forceinline__ void load8(const void* pool, size_t at, float (&x)[8]) {
  if constexpr (kFp8) {
    const uint2 w = *reinterpret_cast<const uint2*>((const uint8_t*)pool + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __builtin_amdgcn_cvt_f32_fp8((int)(w.x >> (8 * i)), 0);
      x[4 + i] = __builtin_amdgcn_cvt_f32_fp8((int)(w.y >> (8 * i)), 0);
    }
  } else {
    Frag16 f;
    f.u = load16((const bf16_t*)pool + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)f.h[i];
  }
}
template <bool kFp8>
__device__ __forceinline__ float load1(const void* pool, size_t at) {
  if constexpr (kFp8) return __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)pool)[at], 0);
  else return (float)((const bf16_t*)pool)[at];
}

// One row by one wave, a lane a key for the logits and D / 64 channels a lane for
// the values: the maximum first, then weights and sums.  Only keys that take part
// are touched, whatever lies in the others.
template <int D, bool kFp8>
__device__ __forceinline__ void attend_row(const ChunkArgs& a, FastDiv by_block, int b, int h,
                                           size_t qrow, int lo, int hi) {
  constexpr int kPer = D / 64;
  const int lane = threadIdx.x & 63;
  const bf16_t* q = a.q + qrow * D;
  const float qs = a.scale * (a.k_scale != nullptr ? a.k_scale[h] : 1.f) * kLog2e;
  const int32_t* table = a.table + (size_t)b * a.max_blocks;
  // Element of the pools where the head's row of position p begins, or -1.
  auto place = [&](int p) -> long long {
    if (p >= hi) return -1;
    const int j = fast_div(p, by_block);
    const int page = table[j];
    if (page < 0 || page >= a.num_blocks) return -1;
    return (((long long)page * a.block_size + (p - j * a.block_size)) * a.H + h) * D;
  };
  auto logit = [&](long long at) {
    float s = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 8) {
      float k[8], x[8];
      load8<kFp8>(a.k_cache, (size_t)at + d, k);
      load8<false>(q, d, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(k[i], x[i], s);
    }
    return s * qs;
  };
  float m = -__builtin_huge_valf();
#pragma unroll 1
  for (int p = lo; p < hi; p += 64) {
    const long long at = place(p + lane);
    if (at >= 0) m = fmaxf(m, logit(at));
  }
  m = wave_reduce(m, [](float x, float y) { return fmaxf(x, y); });
  const float safe = m == -__builtin_huge_valf() ? 0.f : m;
  // Sums that pass the largest number are taken from those of weights 2^-32 as
  // large, which cannot (a row has at most 2^30 keys).
  constexpr float kDown = 0x1p-32f;
  float l = 0.f, o[kPer] = {}, less[kPer] = {};
#pragma unroll 1
  for (int p = lo; p < hi; p += 64) {
    const long long at = place(p + lane);
    const float w = at >= 0 ? __builtin_amdgcn_exp2f(logit(at) - safe) : 0.f;
    l += w;
    for (uint64_t there = __ballot(at >= 0); there != 0; there &= there - 1) {
      const int i = __ffsll((unsigned long long)there) - 1;
      const float wi = __shfl(w, i);
      const size_t from = (size_t)__shfl(at, i) + lane * kPer;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float v = load1<kFp8>(a.v_cache, from + j);
        o[j] = fmaf(wi, v, o[j]);
        less[j] = fmaf(wi * kDown, v, less[j]);
      }
    }
  }
  l = wave_sum(l);
  const float f = l == 0.f ? 0.f : (a.v_scale != nullptr ? a.v_scale[h] : 1.f) / l;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float y = fabsf(o[j]) < __builtin_huge_valf() ? o[j] * f : less[j] * (f / kDown);
    a.out[qrow * D + lane * kPer + j] = (bf16_t)(l == 0.f ? 0.f : y);
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[qrow] = l == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace

// A wave a row and query head.
template <int D, bool kFp8>
__global__ __launch_bounds__(256) void chunk_row_kernel(ChunkArgs a, FastDiv by_block) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long items = (long long)a.T * a.Hq;
  for (long long item = (long long)blockIdx.x * 4 + wave; item < items;
       item += (long long)gridDim.x * 4) {
    const int t = (int)floor_div(item, a.Hq), hq = (int)(item - (long long)t * a.Hq);
    if (t >= min(a.cu_new[a.B], a.T) || t < a.cu_new[0]) continue;
    const int b = __builtin_amdgcn_readfirstlane(last_at_most(a.cu_new, a.B, t));
    const Chunk c = chunk_of(a, b);
    const int i = t - c.row0;
    const int end = i < c.live ? c.at + i + 1 : 0;
    const int lo = a.window > 0 ? max(0, end - a.window) : 0;
    attend_row<D, kFp8>(a, by_block, b, hq / (a.Hq / a.H), (size_t)item, lo, end);
  }
}

size_t chunk_scratch_floats(int T, int B, int Hq, int H, int D) { return 64; }

namespace {

template <int D>
hipError_t launch_chunk(const ChunkArgs& a, hipStream_t stream) {
  const int grid = (int)std::min<long long>(((long long)a.T * a.Hq + 3) / 4, 1 << 16);
  if (a.dtype == kCacheFp8)
    chunk_row_kernel<D, true><<<grid, 256, 0, stream>>>(a, make_fast_div(a.block_size));
  else
    chunk_row_kernel<D, false><<<grid, 256, 0, stream>>>(a, make_fast_div(a.block_size));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_attention(const ChunkArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: return launch_chunk<64>(a, stream);
    case 128: return launch_chunk<128>(a, stream);
    case 256: return launch_chunk<256>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mova

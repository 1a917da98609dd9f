// Attention of one new token per request over the paged key-value cache.
#include <algorithm>

#include "paged.h"

namespace mova {

// Workgroup (query head, request); a wave takes every fourth key.
template <bool kFp8>
__global__ __launch_bounds__(256) void attention_kernel(AttentionArgs a) {
  constexpr int kMaxPer = 4;  // channels a lane: D <= 256
  __shared__ float s_m[4], s_l[4], s_o[4][64 * kMaxPer];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int hq = blockIdx.x, b = blockIdx.y;
  const int h = hq / (a.Hq / a.H);
  const int per = a.D / 64;
  const int len = request_len(a.seq_lens, b, a.max_blocks, a.block_size);
  const int lo = a.window > 0 ? max(0, len - a.window) : 0;
  const int blocks = ceil_div(len, a.block_size);
  const long long total = a.sel != nullptr ? (long long)a.keep * a.block_size : len;
  const float qs = a.scale * (a.k_scale != nullptr ? a.k_scale[h] : 1.f);
  float q[kMaxPer], o[kMaxPer] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < per; ++i) q[i] = (float)a.q[((size_t)b * a.Hq + hq) * a.D + i * 64 + lane];
  float m = -__builtin_huge_valf(), l = 0.f;
  auto elem = [&](const void* pool, size_t at) -> float {
    if constexpr (kFp8) return __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t*)pool)[at], 0);
    else return (float)((const __bf16*)pool)[at];
  };
  for (long long v = wave; v < total; v += 4) {
    int j = (int)(v / a.block_size);
    const int r = (int)(v - (long long)j * a.block_size);
    if (a.sel != nullptr) j = a.sel[((size_t)b * a.H + h) * a.keep + j];
    if (j < 0 || j >= blocks) continue;
    const int p = j * a.block_size + r;
    if (p < lo || p >= len) continue;
    const int page = a.table[(size_t)b * a.max_blocks + j];
    if (page < 0 || page >= a.num_blocks) continue;
    const size_t at = (((size_t)page * a.block_size + r) * a.H + h) * a.D + lane;
    float s = 0.f;
    for (int i = 0; i < per; ++i) s += q[i] * elem(a.k_cache, at + i * 64);
    for (int x = 32; x > 0; x >>= 1) s += __shfl_xor(s, x);
    s *= qs;
    const float mn = fmaxf(m, s);
    const float safe = mn == -__builtin_huge_valf() ? 0.f : mn;
    const float keep = expf(m - safe), p1 = expf(s - safe);
    m = mn;
    l = l * keep + p1;
    for (int i = 0; i < per; ++i) o[i] = o[i] * keep + p1 * elem(a.v_cache, at + i * 64);
  }
  if (lane == 0) { s_m[wave] = m; s_l[wave] = l; }
  for (int i = 0; i < per; ++i) s_o[wave][i * 64 + lane] = o[i];
  __syncthreads();
  const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float safe = M == -__builtin_huge_valf() ? 0.f : M;
  float L = 0.f;
  for (int w = 0; w < 4; ++w) L += s_l[w] * expf(s_m[w] - safe);
  if (threadIdx.x < a.D) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w) x += s_o[w][threadIdx.x] * expf(s_m[w] - safe);
    x = L == 0.f ? 0.f : x / L * (a.v_scale != nullptr ? a.v_scale[h] : 1.f);
    a.out[((size_t)b * a.Hq + hq) * a.D + threadIdx.x] = (__bf16)x;
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[(size_t)b * a.Hq + hq] = L == 0.f ? -__builtin_huge_valf() : safe + logf(L);
}

size_t attention_scratch_floats(int B, int Hq, int H, int D, int max_blocks, int block_size,
                                int keep) {
  (void)Hq; (void)H; (void)D; (void)max_blocks; (void)block_size; (void)keep;
  return B > 0 ? 64 : 0;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream) {
  const dim3 grid(a.Hq, a.B);
  if (a.dtype == kCacheFp8) attention_kernel<true><<<grid, 256, 0, stream>>>(a);
  else attention_kernel<false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mova

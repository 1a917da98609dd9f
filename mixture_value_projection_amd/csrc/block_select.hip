// Block selection for sparse attention: per request and key head, the cache
// blocks whose keys can reach the highest logits.
#include <algorithm>

#include "paged.h"

namespace mova {

namespace {

// The order of the choice as unsigned numbers: a < b as doubles iff
// key(a) < key(b); -0 counts as 0 and NaN as the lowest.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) x = -__builtin_huge_val();
  x += 0.0;
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

}  // namespace

// Wave (b, h, j): score of one block.
__global__ __launch_bounds__(256) void select_score_kernel(SelectArgs a) {
  const int lane = threadIdx.x & 63;
  const int j = blockIdx.x * 4 + (threadIdx.x >> 6), h = blockIdx.y, b = blockIdx.z;
  const int len = request_len(a.seq_lens, b, a.max_blocks, a.block_size);
  if (j >= ceil_div(len, a.block_size)) return;
  const int page = a.table[(size_t)b * a.max_blocks + j];
  const int group = a.Hq / a.H;
  double best = -__builtin_huge_val();
  if (page >= 0 && page < a.num_blocks) {
    const __bf16* lo = a.bounds + ((size_t)page * a.H + h) * 2 * a.D;
    for (int g = 0; g < group; ++g) {
      double s = 0;
      for (int d = lane; d < a.D; d += 64) {
        const double q = (double)(float)a.q[((size_t)b * a.Hq + h * group + g) * a.D + d];
        s += q * (double)(float)(q > 0 ? lo[a.D + d] : lo[d]);
      }
      for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
      if (s > best) best = s;  // NaN never wins
    }
  }
  if (lane == 0) a.scores[((size_t)b * a.H + h) * a.max_blocks + j] = best;
}

// Workgroup (h, b): the `keep` blocks by (forced, score, lower index), in
// index order.
__global__ __launch_bounds__(256) void select_top_kernel(SelectArgs a) {
  __shared__ int hist[256];
  __shared__ unsigned long long s_prefix;
  __shared__ int s_left, s_wave[4];
  const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
  const int n = ceil_div(request_len(a.seq_lens, b, a.max_blocks, a.block_size), a.block_size);
  const double* sc = a.scores + ((size_t)b * a.H + h) * a.max_blocks;
  const int32_t* row = a.table + (size_t)b * a.max_blocks;
  int32_t* sel = a.sel + ((size_t)b * a.H + h) * a.keep;
  // 0: not there (page outside the pool); forced blocks above every score.
  auto key = [&](int j) -> unsigned long long {
    const int page = row[j];
    if (page < 0 || page >= a.num_blocks) return 0ull;
    if (j < a.first || j >= n - a.last) return ~0ull;
    return order_key(sc[j]);
  };
  // The keep-th largest key, digit by digit, and how many equal to it go in.
  if (tid == 0) { s_prefix = 0; s_left = a.keep; }
  __syncthreads();
  for (int shift = 56; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    const unsigned long long prefix = s_prefix;
    for (int j = tid; j < n; j += 256) {
      const unsigned long long k = key(j);
      if (k != 0 && (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8))))
        atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = s_left, d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_left = left;
      s_prefix = prefix | ((unsigned long long)d << shift);
    }
    __syncthreads();
  }
  const unsigned long long cut = s_prefix;
  const int ties = s_left;
  int out = 0, equal = 0;  // chosen, and equal keys seen, before this round
  for (int j0 = 0; j0 < n; j0 += 256) {
    const int j = j0 + tid;
    const unsigned long long k = j < n ? key(j) : 0ull;
    const uint64_t below = (1ull << (tid & 63)) - 1;
    auto rank = [&](bool x, int* sum) {
      const uint64_t m = __ballot(x);
      __syncthreads();
      if ((tid & 63) == 0) s_wave[tid >> 6] = __popcll(m);
      __syncthreads();
      int r = __popcll(m & below);
      for (int w = 0; w < (tid >> 6); ++w) r += s_wave[w];
      *sum = s_wave[0] + s_wave[1] + s_wave[2] + s_wave[3];
      return r;
    };
    int sum;
    const bool eq = k != 0 && k == cut;
    const int er = rank(eq, &sum);
    const bool take = k != 0 && (k > cut || (eq && equal + er < ties));
    equal += sum;
    const int r = rank(take, &sum);
    if (take && out + r < a.keep) sel[out + r] = j;
    out += sum;
  }
  for (int i = out + tid; i < a.keep; i += 256) sel[i] = -1;
}

hipError_t launch_block_select(const SelectArgs& a, hipStream_t stream) {
  select_score_kernel<<<dim3(ceil_div(a.max_blocks, 4), a.H, a.B), 256, 0, stream>>>(a);
  select_top_kernel<<<dim3(a.H, a.B), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mova

// Block selection for sparse attention: per request and key head, the cache
// blocks whose keys can reach the highest logits.
//
// With (lo, hi) the smallest and largest element of each channel over a
// block's keys, no key of the block has a larger logit with q than
//
//   s = sum_d (q_d > 0 ? hi_d : lo_d) q_d,
//
// and a block counts with the largest s of the query heads that share its key
// head.  Two kernels: scores, then the choice.
//
// Scores are bound by reading the bounds, 4 head_dim bytes per block and key
// head against 2 head_dim block_size bytes of keys.  They are 64-bit sums: a
// bf16 product has 16 bits, so the sums are exact but for wide ranges of
// exponents, and the choice does not change with the order of summation.  The
// blocks of the batch form one line in tiles of 16, cut into equal stretches
// as in attention.hip; a wave holds one key head's queries in registers and
// reads 16 bytes of lo and hi a lane.  The 64-bit products run at the rate of
// 32-bit ones on this chip's vector units: about 3 instructions a product.
//
// The choice narrows the range of the order keys (unsigned 64-bit numbers in
// the scores' order) around the keep-th largest: a histogram over 2048 equal
// parts of the range, the part that holds it, and again, until the part's
// keys are all wanted or are equal.  Random scores take two or three rounds.
#include <algorithm>

#include "paged.h"

namespace mova {

namespace {

constexpr int kScoreGrid = 1024;  // 4 workgroups a CU
constexpr int kTileBlocks = 16;
constexpr int kHeadsAtOnce = 4;   // query heads whose 64-bit values a lane holds

constexpr unsigned long long kMissing = 0ull;  // below every score's key
constexpr unsigned long long kForced = ~0ull;  // above every score's key

// a < b as doubles iff key(a) < key(b); -0 counts as 0, NaN as -infinity.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) x = -__builtin_huge_val();
  x += 0.0;
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

template <int kCtrl>
__device__ __forceinline__ double dpp(double x) {
  const uint2 u = __builtin_bit_cast(uint2, x);
  uint2 r;
  r.x = (uint32_t)__builtin_amdgcn_mov_dpp((int)u.x, kCtrl, 0xf, 0xf, true);
  r.y = (uint32_t)__builtin_amdgcn_mov_dpp((int)u.y, kCtrl, 0xf, 0xf, true);
  return __builtin_bit_cast(double, r);
}

// Sum over each run of kLanes (8, 16 or 32) lanes, in all of them.
template <int kLanes>
__device__ __forceinline__ double lanes_sum(double x) {
  x += dpp<0xB1>(x);   // quad_perm 1 0 3 2
  x += dpp<0x4E>(x);   // quad_perm 2 3 0 1
  x += dpp<0x141>(x);  // row_half_mirror
  if constexpr (kLanes >= 16) x += dpp<0x140>(x);  // row_mirror
  if constexpr (kLanes >= 32) x += __shfl_xor(x, 16);
  return x;
}

}  // namespace

template <int D, int kHeads>
__global__ __launch_bounds__(256) void select_score_kernel(SelectArgs a) {
  constexpr int kLanes = D / 8;            // lanes of a block
  constexpr int kAtOnce = 64 / kLanes;     // blocks a wave reads at once
  constexpr int kSteps = kTileBlocks / kAtOnce;
  constexpr int kStripes = 4 / kHeads;
  __shared__ LineShared s_line;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hsub = wave / kStripes, stripe = wave % kStripes;
  const int G = a.Hq / a.H;
  const int groups = a.H / kHeads;
  auto blocks_of = [&](int b) {
    return ceil_div(request_len(a.seq_lens, b, a.max_blocks, a.block_size), a.block_size);
  };
  auto tiles_of = [&](int n) { return ceil_div(n, kTileBlocks * kStripes); };
  Line line;
  if (!line_begin(a.B, [&](int b) { return (long long)tiles_of(blocks_of(b)) * groups; }, s_line,
                  nullptr, &line))
    return;

  int b = line.b;
  long long at = line.first;
  int n = blocks_of(b), tiles = tiles_of(n);
  for (long long pos = line.start; pos < line.end;) {
    while (pos >= at + (long long)tiles * groups) {
      at += (long long)tiles * groups;
      n = blocks_of(++b);
      tiles = tiles_of(n);
    }
    const int hgroup = (int)((pos - at) / tiles);
    const int t0 = (int)(pos - at - (long long)hgroup * tiles);
    const int t1 = (int)min((long long)tiles, t0 + (line.end - pos));
    pos += t1 - t0;
    const int h = hgroup * kHeads + hsub;
    const int32_t* table = a.table + (size_t)b * a.max_blocks;
    unsigned long long* keys = a.keys + ((size_t)b * a.H + h) * a.max_blocks;
    const __bf16* qrow = a.q + ((size_t)b * a.Hq + h * G) * D + (lane % kLanes) * 8;

    double q[kHeadsAtOnce][8];
    auto load_q = [&](int g0) {
#pragma unroll
      for (int g = 0; g < kHeadsAtOnce; ++g) {
        // Heads past the group repeat its last.
        Frag16 f;
        f.u = load16(qrow + (size_t)min(g0 + g, G - 1) * D);
#pragma unroll
        for (int d = 0; d < 8; ++d) q[g][d] = (double)(float)f.h[d];
      }
    };
    load_q(0);
    auto page_of = [&](int x) {
      const int j = (x * kStripes + stripe) * kTileBlocks + (lane & (kTileBlocks - 1));
      const int p = x < t1 && j < n ? table[j] : -1;
      return p < a.num_blocks ? p : -1;
    };
    int next = page_of(t0);
    for (int x = t0; x < t1; ++x) {
      const int page = next;
      next = page_of(x + 1);
      Frag16 lo[kSteps], hi[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int p = max(__shfl(page, u * kAtOnce + lane / kLanes), 0);
        const __bf16* src = a.bounds + ((size_t)p * a.H + h) * 2 * D + (lane % kLanes) * 8;
        lo[u].u = load16_stream(src);
        hi[u].u = load16_stream(src + D);
      }
      double best[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) best[u] = -__builtin_huge_val();
      for (int g0 = 0; g0 < G; g0 += kHeadsAtOnce) {
        if (G > kHeadsAtOnce) load_q(g0);
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          double s[kHeadsAtOnce];
#pragma unroll
          for (int g = 0; g < kHeadsAtOnce; ++g) {
            s[g] = 0;
#pragma unroll
            for (int d = 0; d < 8; ++d)
              s[g] += (double)(q[g][d] > 0 ? (float)hi[u].h[d] : (float)lo[u].h[d]) * q[g][d];
            s[g] = lanes_sum<kLanes>(s[g]);
            best[u] = fmax(best[u], s[g]);  // a NaN does not count
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int i = u * kAtOnce + lane / kLanes;
        const int j = (x * kStripes + stripe) * kTileBlocks + i;
        const int p = __shfl(page, i);
        if (lane % kLanes == 0 && j < n)
          keys[j] = p < 0 ? kMissing
                    : j < a.first || j >= n - a.last ? kForced : order_key(best[u]);
      }
    }
  }
}

// Workgroup (h, b): the `keep` blocks with the highest keys, the lower index
// first among equals, in index order.
constexpr int kTopThreads = 1024;
constexpr int kTopWaves = kTopThreads / 64;
constexpr int kParts = 2048;

__global__ __launch_bounds__(kTopThreads) void select_top_kernel(SelectArgs a) {
  __shared__ int hist[kParts];
  __shared__ unsigned long long s_lo[kTopWaves], s_hi[kTopWaves];
  __shared__ int s_n[kTopWaves], s_f[kTopWaves], s_part, s_above, s_in;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = ceil_div(request_len(a.seq_lens, b, a.max_blocks, a.block_size), a.block_size);
  const unsigned long long* keys = a.keys + ((size_t)b * a.H + h) * a.max_blocks;
  int32_t* sel = a.sel + ((size_t)b * a.H + h) * a.keep;

  // How many are there and forced, and the range of the others' keys.
  unsigned long long lo = ~0ull, hi = 0;
  int there = 0, forced = 0;
  for (int j = tid; j < n; j += kTopThreads) {
    const unsigned long long k = keys[j];
    there += k != kMissing;
    forced += k == kForced;
    if (k != kMissing && k != kForced) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    lo = min(lo, (unsigned long long)__shfl_xor((long long)lo, o));
    hi = max(hi, (unsigned long long)__shfl_xor((long long)hi, o));
    there += __shfl_xor(there, o);
    forced += __shfl_xor(forced, o);
  }
  if (lane == 0) {
    s_lo[wave] = lo;
    s_hi[wave] = hi;
    s_n[wave] = there;
    s_f[wave] = forced;
  }
  __syncthreads();
  there = forced = 0;
#pragma unroll
  for (int w = 0; w < kTopWaves; ++w) {
    lo = min(lo, s_lo[w]);
    hi = max(hi, s_hi[w]);
    there += s_n[w];
    forced += s_f[w];
  }

  // Keys from `cut` on are taken; of those equal to it, the first `ties`.
  unsigned long long cut = 1;
  int ties = n;
  if (there > a.keep) {
    int left = a.keep - forced;  // wanted of the keys in [lo, hi]
    if (left <= 0) {
      cut = kForced;
      ties = a.keep;
    } else {
      for (;;) {
        const unsigned long long span = hi - lo;
        const int bits = span == 0 ? 0 : 64 - __clzll((long long)span);
        const int shift = max(bits - 11, 0);
        hist[tid] = 0;
        hist[tid + kTopThreads] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += kTopThreads) {
          const unsigned long long k = keys[j];
          if (k >= lo && k <= hi && k != kMissing) atomicAdd(&hist[(k - lo) >> shift], 1);
        }
        __syncthreads();
        // Counts from the top: each thread two parts, then over the waves.
        const int p1 = kParts - 1 - 2 * tid, p0 = p1 - 1;
        const int c1 = hist[p1], c0 = hist[p0];
        int inc = c1 + c0;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int up = __shfl_up(inc, o);
          if (lane >= o) inc += up;
        }
        if (lane == 63) s_n[wave] = inc;
        __syncthreads();
        int above = inc - c1 - c0;
        for (int w = 0; w < wave; ++w) above += s_n[w];
        if (above < left && left <= above + c1) {
          s_part = p1, s_above = above, s_in = c1;
        } else if (above + c1 < left && left <= above + c1 + c0) {
          s_part = p0, s_above = above + c1, s_in = c0;
        }
        __syncthreads();
        left -= s_above;
        lo += (unsigned long long)s_part << shift;
        if (shift == 0 || s_in == left) {
          cut = lo;
          ties = shift == 0 ? left : n;
          break;
        }
        hi = min(hi, lo + ((1ull << shift) - 1));
      }
    }
  }

  // Taken blocks before each, counted per wave and round in index order.
  int out = 0, seen = 0;
  for (int j0 = 0; j0 < n; j0 += kTopThreads) {
    const int j = j0 + tid;
    const unsigned long long k = j < n ? keys[j] : kMissing;
    const uint64_t above = __ballot(k > cut), equal = __ballot(k == cut && k != kMissing);
    const uint64_t before = (1ull << lane) - 1;
    __syncthreads();
    if (lane == 0) {
      s_n[wave] = __popcll(above);
      s_f[wave] = __popcll(equal);
    }
    __syncthreads();
    int r = out + __popcll(above & before), e = seen + __popcll(equal & before);
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w) {
      if (w < wave) {
        r += s_n[w];
        e += s_f[w];
      }
      out += s_n[w];
      seen += s_f[w];
    }
    const bool take = k > cut || (k == cut && k != kMissing && e < ties);
    if (take) sel[r + min(e, ties)] = j;
  }
  for (int i = out + min(seen, ties) + tid; i < a.keep; i += kTopThreads) sel[i] = -1;
}

hipError_t launch_block_select(const SelectArgs& a, hipStream_t stream) {
  const int heads = a.H % 4 == 0 ? 4 : a.H % 2 == 0 ? 2 : 1;
  auto score = [&](auto kernel) { kernel<<<kScoreGrid, 256, 0, stream>>>(a); };
  switch (a.D) {
    case 64:
      heads == 4   ? score(select_score_kernel<64, 4>)
      : heads == 2 ? score(select_score_kernel<64, 2>)
                   : score(select_score_kernel<64, 1>);
      break;
    case 128:
      heads == 4   ? score(select_score_kernel<128, 4>)
      : heads == 2 ? score(select_score_kernel<128, 2>)
                   : score(select_score_kernel<128, 1>);
      break;
    case 256:
      heads == 4   ? score(select_score_kernel<256, 4>)
      : heads == 2 ? score(select_score_kernel<256, 2>)
                   : score(select_score_kernel<256, 1>);
      break;
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  select_top_kernel<<<dim3(a.H, a.B), kTopThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mova

// Block selection for sparse attention: per request and key head, the cache
// blocks whose keys can reach the highest logits.
//
// With (lo, hi) the smallest and largest element of each channel over a
// block's keys, no key of the block has a larger logit with q than
//
//   s = sum_d (q_d > 0 ? hi_d : lo_d) q_d = sum_d hi_d q+_d + lo_d q-_d
//
// (q+ and q- the positive and negative parts), and a block counts with the
// largest s of the query heads that share its key head.  The choice is that of
// the 64-bit sums: a bf16 product has 16 bits, so those are exact but for wide
// ranges of exponents, and it does not change with the order of summation.
//
// Two kernels.  The first encloses every score: MFMA products give
// hi q+ + (-lo) |q-| for 16 blocks and 16 query heads at a time, and a second
// product of the absolute values the error that 32-bit sums can have made.
// That is a few percent of the matrix units, where 64-bit products of every
// block kept the vector units busy for twice the time that the bounds take to
// read (3 requests of 100k to 400k tokens: 42 us; 96 MB of bounds).  The blocks
// of the batch form one line in tiles of 16, cut into equal stretches as in
// attention.hip.
//
// The second kernel finds, per request and key head, the keep-th largest lower
// end, takes the blocks whose upper end reaches it -- a few more than `keep`
// -- and computes only those in 64 bits, unless there are exactly as many as
// wanted.  A histogram over 2048 equal parts of the ends' range narrows the
// search to one part, and again, until the part's blocks are all wanted or are
// equal.
#include <algorithm>
#include <type_traits>

#include "paged.h"

namespace mova {

namespace {

constexpr int kScoreGrid = 1024;  // 4 workgroups a CU
constexpr int kTileBlocks = 16;

// Bound on the error of a 32-bit sum s of products with absolute sum t, in any
// order of summation, the additions rounded or cut: at most 2 * 256 products
// lose 2^-23 t each (2^-14 t), a quarter of this; products below the smallest
// number at most 2^-140 together.
constexpr float kErrorRel = 1.f / 4096;
constexpr float kErrorAbs = 7.5e-37f;  // 2^-120

// [lower, upper] of a block's score.  Missing blocks: upper = -infinity;
// blocks that are always in: lower = +infinity; a score that 32 bits cannot
// enclose: (-infinity, +infinity).
struct Interval {
  float lower, upper;
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr unsigned long long kMissing = 0ull;  // below every score's key
constexpr unsigned long long kForced = ~0ull;  // above every score's key

// a < b as doubles iff key(a) < key(b); -0 counts as 0, NaN as -infinity.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) x = -__builtin_huge_val();
  x += 0.0;
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// Largest over each run of 16 lanes, in all of them.
__device__ __forceinline__ float max16(float x) {
  auto other = [&](auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x),
                                                              decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x = fmaxf(x, other(std::integral_constant<int, 0xB1>{}));   // quad_perm 1 0 3 2
  x = fmaxf(x, other(std::integral_constant<int, 0x4E>{}));   // quad_perm 2 3 0 1
  x = fmaxf(x, other(std::integral_constant<int, 0x141>{}));  // row_half_mirror
  return fmaxf(x, other(std::integral_constant<int, 0x140>{}));  // row_mirror
}

__device__ __forceinline__ int blocks_of(const SelectArgs& a, int b) {
  return a.num_blocks > 0
             ? ceil_div(request_len(a.seq_lens, b, a.max_blocks, a.block_size), a.block_size)
             : 0;
}

}  // namespace

// kHeads: key heads of a workgroup; 4 / kHeads waves share a head's tiles.
// MFMA rows are blocks, columns query heads (those past the group are left
// out of the maxima).
template <int D, int kHeads>
__global__ __launch_bounds__(256) void select_score_kernel(SelectArgs a) {
  constexpr int kStripes = 4 / kHeads;
  constexpr int kSteps = D / 32;
  __shared__ LineShared s_line;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int hsub = wave / kStripes, stripe = wave % kStripes;
  const int G = a.Hq / a.H;
  const int groups = a.H / kHeads;
  auto tiles_of = [&](int n) { return ceil_div(n, kTileBlocks * kStripes); };
  Line line;
  if (!line_begin(a.B, [&](int b) { return (long long)tiles_of(blocks_of(a, b)) * groups; }, s_line,
                  nullptr, &line))
    return;

  int b = line.b;
  long long at = line.first;
  int n = blocks_of(a, b), tiles = tiles_of(n);
  for (long long pos = line.start; pos < line.end;) {
    while (pos >= at + (long long)tiles * groups) {
      at += (long long)tiles * groups;
      n = blocks_of(a, ++b);
      tiles = tiles_of(n);
    }
    const int hgroup = (int)((pos - at) / tiles);
    const int t0 = (int)(pos - at - (long long)hgroup * tiles);
    const int t1 = (int)min((long long)tiles, t0 + (line.end - pos));
    pos += t1 - t0;
    const int h = hgroup * kHeads + hsub;
    const int32_t* table = a.table + (size_t)b * a.max_blocks;
    Interval* out = (Interval*)a.scratch + ((size_t)b * a.H + h) * a.max_blocks;

    // q+ and |q-| of query head g0 + r16 as MFMA columns.
    Frag16 qp[kSteps], qn[kSteps];
    auto load_q = [&](int g0) {
      const __bf16* row = a.q + ((size_t)b * a.Hq + h * G + min(g0 + r16, G - 1)) * D + 8 * g4;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        Frag16 f;
        f.u = load16(row + 32 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // Bits of the elements whose sign is set.
          const uint32_t neg = ((f.u[i] & 0x80008000u) >> 15) * 0xffffu;
          qp[u].u[i] = f.u[i] & ~neg;
          qn[u].u[i] = f.u[i] & neg & 0x7fff7fffu;
        }
      }
    };
    load_q(0);
    auto page_of = [&](int x) {
      const int j = (x * kStripes + stripe) * kTileBlocks + r16;
      const int p = x < t1 && j < n ? table[j] : -1;
      return p < a.num_blocks ? p : -1;
    };
    int next = page_of(t0);
    for (int x = t0; x < t1; ++x) {
      const int page = next;
      next = page_of(x + 1);
      const __bf16* src = a.bounds + ((size_t)max(page, 0) * a.H + h) * 2 * D + 8 * g4;
      Frag16 lo[kSteps], hi[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        lo[u].u = load16_stream(src + 32 * u);
        hi[u].u = load16_stream(src + D + 32 * u);
      }
      Interval best[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) best[i] = {-__builtin_huge_valf(), -__builtin_huge_valf()};
      for (int g0 = 0; g0 < G; g0 += 16) {
        if (G > 16) load_q(g0);
        f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f}, t = s;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          Frag16 x0, x1;
          s = mfma16x16x32(hi[u].h, qp[u].h, s);
          x0.u = lo[u].u ^ 0x80008000u;
          s = mfma16x16x32(x0.h, qn[u].h, s);
          x0.u = hi[u].u & 0x7fff7fffu;
          x1.u = lo[u].u & 0x7fff7fffu;
          t = mfma16x16x32(x0.h, qp[u].h, t);
          t = mfma16x16x32(x1.h, qn[u].h, t);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = t[i] * kErrorRel + kErrorAbs;
          const bool enclosed = fabsf(s[i]) + t[i] < 3e38f;
          float lower = enclosed ? s[i] - e : -__builtin_huge_valf();
          float upper = enclosed ? s[i] + e : __builtin_huge_valf();
          if (g0 + r16 >= G) lower = upper = -__builtin_huge_valf();
          best[i].lower = fmaxf(best[i].lower, lower);
          best[i].upper = fmaxf(best[i].upper, upper);
        }
      }
      Interval mine = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Interval v = {max16(best[i].lower), max16(best[i].upper)};
        if (r16 == i) mine = v;
      }
      const int i = 4 * g4 + (r16 & 3);
      const int j = (x * kStripes + stripe) * kTileBlocks + i;
      const int p = __shfl(page, i);
      if (r16 < 4 && j < n) {
        if (p < 0) mine = {-__builtin_huge_valf(), -__builtin_huge_valf()};
        else if (j < a.first || j >= n - a.last) mine = {__builtin_huge_valf(), __builtin_huge_valf()};
        out[j] = mine;
      }
    }
  }
}

namespace {

constexpr int kTopThreads = 1024;
constexpr int kTopWaves = kTopThreads / 64;
constexpr int kParts = 2048;
constexpr int kHeld = 16;              // intervals a thread holds at a time
constexpr int kMaxCandidates = 1024;   // computed in LDS; beyond, in memory

struct TopShared {
  int hist[kParts];
  unsigned long long key[kMaxCandidates];
  int block[kMaxCandidates];
  int count[kHeld][kTopWaves];
  unsigned long long lo[kTopWaves], hi[kTopWaves];
  int n[kTopWaves], f[kTopWaves];
  int part, above, in;
};

template <class K>
__device__ __forceinline__ K wave_min(K x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = min(x, (K)__shfl_xor((long long)x, o));
  return x;
}
template <class K>
__device__ __forceinline__ K wave_max(K x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = max(x, (K)__shfl_xor((long long)x, o));
  return x;
}
__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Narrows [lo, hi] around the left-th largest of the keys in it, which
// for_each(f) hands to f one after the other.  Returns the cut: keys from it
// on are wanted, and of those equal to it the first *ties.
template <class K, class ForEach>
__device__ K narrow(TopShared& sh, K lo, K hi, int left, ForEach for_each, int* ties) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (;;) {
    const unsigned long long span = (unsigned long long)(hi - lo);
    const int bits = span == 0 ? 0 : 64 - __clzll((long long)span);
    const int shift = max(bits - 11, 0);
    sh.hist[tid] = 0;
    sh.hist[tid + kTopThreads] = 0;
    __syncthreads();
    for_each([&](K k) {
      if (k >= lo && k <= hi) atomicAdd(&sh.hist[(int)((k - lo) >> shift)], 1);
    });
    __syncthreads();
    // Counts from the top: each thread two parts, then over the waves.
    const int p1 = kParts - 1 - 2 * tid, p0 = p1 - 1;
    const int c1 = sh.hist[p1], c0 = sh.hist[p0];
    int inc = c1 + c0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 63) sh.n[wave] = inc;
    __syncthreads();
    int above = inc - c1 - c0;
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w)
      if (w < wave) above += sh.n[w];
    if (above < left && left <= above + c1) {
      sh.part = p1;
      sh.above = above;
      sh.in = c1;
    } else if (above + c1 < left && left <= above + c1 + c0) {
      sh.part = p0;
      sh.above = above + c1;
      sh.in = c0;
    }
    __syncthreads();
    left -= sh.above;
    lo += (K)((K)sh.part << shift);
    if (shift == 0 || sh.in == left) {
      *ties = shift == 0 ? left : 0x7fffffff;
      return lo;
    }
    hi = min(hi, (K)(lo + (K)(((K)1 << shift) - 1)));
  }
}

// 64-bit score of a block, in each of 16 lanes that work on it.
__device__ __forceinline__ double exact_score(const SelectArgs& a, int b, int h, int page, int l) {
  const int G = a.Hq / a.H;
  const __bf16* lo = a.bounds + ((size_t)page * a.H + h) * 2 * a.D;
  double best = -__builtin_huge_val();
  for (int g = 0; g < G; ++g) {
    const __bf16* q = a.q + ((size_t)b * a.Hq + h * G + g) * a.D;
    double s = 0;
    for (int d = 4 * l; d < a.D; d += 64) {
      typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
      const bf16x4 qv = *(const bf16x4*)(q + d), lv = *(const bf16x4*)(lo + d),
                   hv = *(const bf16x4*)(lo + a.D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double x = (double)(float)qv[i];
        s += (double)(x > 0 ? (float)hv[i] : (float)lv[i]) * x;
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (s > best) best = s;  // a NaN does not count
  }
  return best;
}

}  // namespace

// Workgroup (h, b): the `keep` blocks with the highest scores, the lower index
// first among equals, in index order.
__global__ __launch_bounds__(kTopThreads) void select_top_kernel(SelectArgs a) {
  __shared__ TopShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = blocks_of(a, b);
  const int32_t* table = a.table + (size_t)b * a.max_blocks;
  unsigned long long* scratch = a.scratch + ((size_t)b * a.H + h) * a.max_blocks;
  const Interval* ends = (const Interval*)scratch;
  int32_t* sel = a.sel + ((size_t)b * a.H + h) * a.keep;
  const float inf = __builtin_huge_valf();

  // A thread holds kHeld intervals, of blocks base + i * kTopThreads + tid;
  // lists that need more are read again in each pass.
  Interval iv[kHeld];
  auto hold = [&](int base) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int j = base + i * kTopThreads + tid;
      iv[i] = j < n ? ends[j] : Interval{-inf, -inf};
    }
  };
  auto for_each = [&](auto f) {
    for (int base = 0; base < n; base += kHeld * kTopThreads) {
      if (n > kHeld * kTopThreads) hold(base);
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (base + i * kTopThreads < n) f(iv[i]);
    }
  };
  hold(0);
  auto regular = [&](const Interval& v) { return v.upper > -inf && v.lower < inf; };

  uint32_t lo = ~0u, hi = 0;
  int there = 0, forced = 0;
  for_each([&](const Interval& v) {
    there += v.upper > -inf;
    forced += v.lower == inf;
    if (regular(v)) {
      lo = min(lo, order_key(v.lower));
      hi = max(hi, order_key(v.lower));
    }
  });
  lo = wave_min(lo);
  hi = wave_max(hi);
  there = wave_sum(there);
  forced = wave_sum(forced);
  if (lane == 0) {
    sh.lo[wave] = lo;
    sh.hi[wave] = hi;
    sh.n[wave] = there;
    sh.f[wave] = forced;
  }
  __syncthreads();
  there = forced = 0;
#pragma unroll
  for (int w = 0; w < kTopWaves; ++w) {
    lo = min(lo, (uint32_t)sh.lo[w]);
    hi = max(hi, (uint32_t)sh.hi[w]);
    there += sh.n[w];
    forced += sh.f[w];
  }
  __syncthreads();

  // Blocks whose score may be among the wanted: all, none (the forced ones
  // fill the list), or those that reach the left-th largest lower end.
  const int left = min(a.keep, there) - forced;
  uint32_t reach = 0;
  if (left <= 0) {
    reach = ~0u;
  } else if (there > a.keep) {
    int ties;
    reach = narrow(sh, lo, hi, left, [&](auto f) {
      for_each([&](const Interval& v) { if (regular(v)) f(order_key(v.lower)); });
    }, &ties);
  }
  auto candidate = [&](const Interval& v) { return regular(v) && order_key(v.upper) >= reach; };
  int candidates = 0;
  for_each([&](const Interval& v) { candidates += candidate(v); });
  candidates = wave_sum(candidates);
  if (lane == 0) sh.f[wave] = candidates;
  __syncthreads();
  candidates = 0;
#pragma unroll
  for (int w = 0; w < kTopWaves; ++w) candidates += sh.f[w];

  const uint64_t below = (1ull << lane) - 1;
  // Calls put(i, rank) for the held intervals that `is` picks, ranked in index
  // order from `from` on; returns the next rank.
  auto ranked = [&](auto is, int from, auto put) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint64_t m = __ballot(is(iv[i]));
      if (lane == 0) sh.count[i][wave] = __popcll(m);
    }
    __syncthreads();
    // The 256 counts lie in index order; the first wave adds them up.
    if (wave == 0) {
      int* c = &sh.count[0][0] + 4 * lane;
      const int c0 = c[0], c1 = c[1], c2 = c[2], c3 = c[3];
      int inc = c0 + c1 + c2 + c3;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 63) sh.n[0] = inc;
      inc -= c1 + c2 + c3 + c0;
      c[0] = inc;
      c[1] = inc + c0;
      c[2] = inc + c0 + c1;
      c[3] = inc + c0 + c1 + c2;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const bool yes = is(iv[i]);
      const uint64_t m = __ballot(yes);
      if (yes) put(i, from + sh.count[i][wave] + __popcll(m & below));
    }
    return from + sh.n[0];
  };

  if (candidates == max(left, 0)) {
    // Everything that may be wanted is.
    int out = 0;
    for (int base = 0; base < n; base += kHeld * kTopThreads) {
      if (n > kHeld * kTopThreads) hold(base);
      out = ranked([&](const Interval& v) { return v.lower == inf || candidate(v); }, out,
                   [&](int i, int r) { sel[r] = base + i * kTopThreads + tid; });
    }
    for (int i = out + tid; i < a.keep; i += kTopThreads) sel[i] = -1;
    return;
  }
  if (candidates <= kMaxCandidates) {
    // Listed in LDS, computed by 16 lanes each, and chosen by counting the
    // better ones.  Forced blocks are the first and last ones.
    int listed = 0, early = 0;
    for (int base = 0; base < n; base += kHeld * kTopThreads) {
      if (n > kHeld * kTopThreads) hold(base);
      listed = ranked(candidate, listed,
                      [&](int i, int r) { sh.block[r] = base + i * kTopThreads + tid; });
    }
    for (int j = tid; j < min(a.first, n); j += kTopThreads) early += ends[j].lower == inf;
    early = wave_sum(early);
    if (lane == 0) sh.n[wave] = early;
    __syncthreads();
    early = 0;
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w) early += sh.n[w];
    for (int c = tid / 16; c < candidates; c += kTopThreads / 16) {
      const double s = exact_score(a, b, h, table[sh.block[c]], tid & 15);
      if ((tid & 15) == 0) sh.key[c] = order_key(s);
    }
    __syncthreads();
    bool taken = false;
    if (tid < candidates) {
      const unsigned long long k = sh.key[tid];
      int better = 0;
      for (int c = 0; c < candidates; ++c) better += sh.key[c] > k || (sh.key[c] == k && c < tid);
      taken = better < left;
    }
    const uint64_t m = __ballot(taken);
    if (lane == 0) sh.f[wave] = __popcll(m);
    __syncthreads();
    int r = early + __popcll(m & below);
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w)
      if (w < wave) r += sh.f[w];
    if (taken) sel[r] = sh.block[tid];
    // The forced ones in front and behind.
    int front = 0, back = early + left;
    const int late = max(n - a.last, min(a.first, n));
    for (int j0 = 0; j0 < min(a.first, n); j0 += 64) {
      const bool f = j0 + lane < min(a.first, n) && ends[j0 + lane].lower == inf;
      const uint64_t fm = __ballot(f);
      if (f && wave == 0) sel[front + __popcll(fm & below)] = j0 + lane;
      front += __popcll(fm);
    }
    for (int j0 = late; j0 < n; j0 += 64) {
      const bool f = j0 + lane < n && ends[j0 + lane].lower == inf;
      const uint64_t fm = __ballot(f);
      if (f && wave == 0) sel[back + __popcll(fm & below)] = j0 + lane;
      back += __popcll(fm);
    }
    for (int i = back + tid; i < a.keep; i += kTopThreads) sel[i] = -1;
    return;
  }

  // Many candidates (equal scores, long lists): 64-bit keys in place of the
  // intervals, then the same narrowing on them.
  for (int j = tid / 16; j < n; j += kTopThreads / 16) {
    const Interval v = ends[j];
    unsigned long long k = v.lower == inf ? kForced : kMissing;
    if (candidate(v)) k = order_key(exact_score(a, b, h, table[j], tid & 15));
    // The 16 lanes have all read v (they run together) before one writes.
    if ((tid & 15) == 0) scratch[j] = k;
  }
  __syncthreads();
  unsigned long long klo = ~0ull, khi = 0;
  for (int j = tid; j < n; j += kTopThreads) {
    const unsigned long long k = scratch[j];
    if (k != kMissing && k != kForced) {
      klo = min(klo, k);
      khi = max(khi, k);
    }
  }
  klo = wave_min(klo);
  khi = wave_max(khi);
  if (lane == 0) {
    sh.lo[wave] = klo;
    sh.hi[wave] = khi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopWaves; ++w) {
    klo = min(klo, sh.lo[w]);
    khi = max(khi, sh.hi[w]);
  }
  int ties;
  const unsigned long long cut = narrow(sh, klo, khi, left, [&](auto f) {
    for (int j = tid; j < n; j += kTopThreads) f(scratch[j]);
  }, &ties);
  int out = 0, seen = 0;
  for (int j0 = 0; j0 < n; j0 += kTopThreads) {
    const int j = j0 + tid;
    const unsigned long long k = j < n ? scratch[j] : kMissing;
    const uint64_t above = __ballot(k > cut), equal = __ballot(k == cut);
    __syncthreads();
    if (lane == 0) {
      sh.n[wave] = __popcll(above);
      sh.f[wave] = __popcll(equal);
    }
    __syncthreads();
    int r = out + __popcll(above & below), e = seen + __popcll(equal & below);
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w) {
      if (w < wave) {
        r += sh.n[w];
        e += sh.f[w];
      }
      out += sh.n[w];
      seen += sh.f[w];
    }
    if (k > cut || (k == cut && e < ties)) sel[r + min(e, ties)] = j;
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

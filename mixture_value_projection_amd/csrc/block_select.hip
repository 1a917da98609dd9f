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
// read (3 requests of 100k to 400k tokens: 42 us; 125 MB of bounds).  The blocks
// of the batch form one line in tiles of 16, cut into equal stretches as in
// attention.hip.
//
// The second kernel finds, per request and key head, the keep-th largest lower
// end.  A block whose upper end stays below it is out, one whose lower end is
// above every upper end that may still come in from below is in, and the few
// between are computed in 64 bits.  A histogram over 2048 equal parts of the
// ends' range narrows the search to one part, and again, until the part's
// blocks are all wanted or are equal.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "paged.h"

namespace mova {

namespace {

constexpr int kCus = 256;
constexpr int kTileBlocks = kSelectTile;

// Bound on the error of a 32-bit sum s of products with absolute sum t, in any
// order of summation, the additions rounded or cut: at most 2 * 256 products
// lose 2^-23 t each (2^-14 t), a quarter of this; products below the smallest
// number at most 2^-140 together.
constexpr float kErrorRel = 1.f / 4096;
constexpr float kErrorAbs = 7.5e-37f;  // 2^-120

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// The order keys of the ends of a block's score, neither of them 0 or ~0; a
// score that 32 bits cannot enclose has those of -infinity and +infinity.
// Missing blocks: {0, 0}; blocks that are always in: {~0, ~0}.
struct Ends {
  uint32_t lower, upper;
};

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

// Largest over the wave's lanes 16 g + r, r < 4, for all.
__device__ __forceinline__ uint32_t tile_max(uint32_t x) {
  x = max(x, (uint32_t)dpp_or_0<0xB1>((int)x));  // quad_perm 1 0 3 2, 2 3 0 1
  x = max(x, (uint32_t)dpp_or_0<0x4E>((int)x));
  return max(max((uint32_t)read_lane((int)x, 0), (uint32_t)read_lane((int)x, 16)),
             max((uint32_t)read_lane((int)x, 32), (uint32_t)read_lane((int)x, 48)));
}

__device__ __forceinline__ int blocks_of(const SelectArgs& a, int b) {
  return a.num_blocks > 0
             ? ceil_div(request_len(a.seq_lens, b, a.max_blocks, a.block_size), a.block_size)
             : 0;
}

}  // namespace

// kHeads: key heads of a workgroup; 4 / kHeads waves share a head's tiles.
// MFMA rows are blocks, columns query heads (those past the group are left
// out of the maxima).  Each wave reads through a ring of tiles in LDS, as in
// attention.hip: with the fragments read straight into registers, one tile
// ahead or none, the kernel took 40 and 35 us where this takes 25 (3 requests
// of 100k to 400k tokens).
template <int D>
struct BoundsTile {
  static constexpr int kRow = 4 * D;  // bytes of a block's bounds, lo then hi
  static constexpr int kChunks = kRow / 16;
  static constexpr int kRowsPerLoad = 64 / kChunks;
  static constexpr int kBytes = kTileBlocks * kRow;
  static constexpr int kLoads = kTileBlocks / kRowsPerLoad;
  // Two workgroups a CU with 16 KB of bounds a wave, where that is two tiles,
  // or one with 32 (128 wide: 28.9 against 31.5 us for both kernels, 32 requests
  // of up to 30k tokens).
  static constexpr int kPerCu = 2 * kBytes <= 16384 ? 2 : 1;
  static constexpr int kRing = 32768 / kPerCu;
  static constexpr int kStages = kRing / kBytes;
  static constexpr int kLds = kRing + kStages * 256;
};

template <int D, int kHeads>
__global__ __launch_bounds__(256) void select_score_kernel(SelectArgs a) {
  using T = BoundsTile<D>;
  constexpr int kStripes = 4 / kHeads;
  constexpr int kSteps = D / 32;
  constexpr int S = T::kStages;
  constexpr int kGroupLoads = T::kLoads + 1;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
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

  char* ring = lds + wave * T::kLds;
  int* fetched = (int*)(ring + T::kRing);
  int b = line.b;
  long long at = line.first;
  int n = blocks_of(a, b), tiles = tiles_of(n);
  for (long long pos = line.start; pos < line.end;) {
    while (pos >= at + (long long)tiles * groups) {
      at += (long long)tiles * groups;
      if (++b >= a.B) return;
      n = blocks_of(a, b);
      tiles = tiles_of(n);
    }
    const int hgroup = (int)floor_div(pos - at, tiles);
    const int t0 = (int)(pos - at - (long long)hgroup * tiles);
    const int t1 = (int)min((long long)tiles, t0 + (line.end - pos));
    pos += t1 - t0;
    const int h = hgroup * kHeads + hsub;
    const int32_t* table = a.table + (size_t)b * a.max_blocks;
    Ends* out = (Ends*)a.scratch + ((size_t)b * a.H + h) * select_stride(a.max_blocks);
    Ends* tops = (Ends*)a.scratch + select_tiles_at(a.B, a.H, a.max_blocks) +
                 ((size_t)b * a.H + h) * ceil_div(a.max_blocks, kTileBlocks);

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
          const uint32_t m = ((f.u[i] & 0x80008000u) >> 15) * 0xffffu;  // the negative ones
          qp[u].u[i] = f.u[i] & ~m;
          qn[u].u[i] = f.u[i] & m & 0x7fff7fffu;
        }
      }
    };
    load_q(0);
    // Table entry of the lane's block of tile x (a lane a block).
    const int nt = t1 - t0;
    auto block_at = [&](int x) { return ((t0 + x) * kStripes + stripe) * kTileBlocks + r16; };
    auto address = [&](int x) { return table + min(block_at(x), a.max_blocks - 1); };
    // Issues the loads of tile x and the fetch of the table entries of tile
    // x + S; returns the lane's block number, -1 where there is none.
    auto issue = [&](int x, int page) {
      if (block_at(x) >= n || page < 0 || page >= a.num_blocks) page = -1;
      const int row = max(page, 0);
      char* stage = ring + (x & (S - 1)) * T::kBytes;
      constexpr int kUnroll = T::kLoads > 8 ? 4 : T::kLoads;  // fewer addresses at a time
#pragma unroll kUnroll
      for (int i = 0; i < T::kLoads; ++i) {
        const int rr = i * T::kRowsPerLoad + lane / T::kChunks;
        const int c = (lane % T::kChunks) ^ rr;
        piece_to_lds<true>((const char*)a.bounds +
                               ((size_t)(uint32_t)__shfl(row, rr) * a.H + h) * T::kRow + c * 16,
                           stage + i * 1024);
      }
      word_to_lds(address(x + S), fetched + (x & (S - 1)) * 64);
      return page;
    };
    int pages[S] = {};  // of the tiles in the ring, the lane's block of each
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
    asm volatile("" ::: "memory");
#pragma unroll 1
    for (int i = 0; i < S; ++i) word_to_lds(address(i), fetched + i * 64);
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));
    asm volatile("" ::: "memory");
    // The S turns before tile 0 only fill the ring.
    for (int x = -S; x < nt; ++x) {
      const int page = pages[0];
#pragma unroll
      for (int i = 0; i + 1 < S; ++i) pages[i] = pages[i + 1];
      if (x >= 0) {
        wait_groups<S - 1, kGroupLoads>(min(S - 1, nt - 1 - x));
        asm volatile("" ::: "memory");
        const char* stage = ring + (x & (S - 1)) * T::kBytes;
        float lowest[4], highest[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) lowest[i] = highest[i] = -__builtin_huge_valf();
        for (int g0 = 0; g0 < G; g0 += 16) {
          if (G > 16) {
            load_q(g0);
            // Waited for here: a group of up to 16 has no such wait.
#pragma unroll
            for (int u = 0; u < kSteps; ++u) loaded(qp[u].u), loaded(qn[u].u);
          }
          f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f}, t = s;
#pragma unroll
          for (int u = 0; u < kSteps; ++u) {
            Frag16 lo, hi, f;
            lo.u = *reinterpret_cast<const u32x4*>(stage + r16 * T::kRow + ((4 * u + g4) ^ r16) * 16);
            hi.u = *reinterpret_cast<const u32x4*>(stage + r16 * T::kRow +
                                                   ((T::kChunks / 2 + 4 * u + g4) ^ r16) * 16);
            s = mfma16x16x32(hi.h, qp[u].h, s);
            f.u = lo.u ^ 0x80008000u;
            s = mfma16x16x32(f.h, qn[u].h, s);
            f.u = hi.u & 0x7fff7fffu;
            t = mfma16x16x32(f.h, qp[u].h, t);
            f.u = lo.u & 0x7fff7fffu;
            t = mfma16x16x32(f.h, qn[u].h, t);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = t[i] * kErrorRel + kErrorAbs;
            const bool enclosed = fabsf(s[i]) + t[i] < 3e38f;
            float lower = enclosed ? s[i] - e : -__builtin_huge_valf();
            float upper = enclosed ? s[i] + e : __builtin_huge_valf();
            if (g0 + r16 >= G) lower = upper = -__builtin_huge_valf();
            lowest[i] = fmaxf(lowest[i], lower);
            highest[i] = fmaxf(highest[i], upper);
          }
        }
        Ends mine = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Ends v = {order_key(max16(lowest[i])), order_key(max16(highest[i]))};
          if (r16 == i) mine = v;
        }
        const int i = 4 * g4 + (r16 & 3);
        const int j = ((t0 + x) * kStripes + stripe) * kTileBlocks + i;
        const int p = __shfl(page, i);
        if (r16 < 4 && j < n) {
          if (p < 0) mine = {0u, 0u};
          else if (j < a.first || j >= n - a.last) mine = {~0u, ~0u};
          out[j] = mine;
        }
        // The tile's largest ends, of the blocks that are neither missing nor
        // always in.
        const bool counts = r16 < 4 && j < n && mine.lower != ~0u;
        const Ends most = {tile_max(counts ? mine.lower : 0u), tile_max(counts ? mine.upper : 0u)};
        const int tile = (t0 + x) * kStripes + stripe;
        if (lane == 0 && tile * kTileBlocks < n) tops[tile] = most;
      }
      if (x + S < nt) {
        const int entry = fetched[(x & (S - 1)) * 64 + lane];
        __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
        asm volatile("" ::: "memory");
        pages[S - 1] = issue(x + S, entry);
      }
    }
  }
}

namespace {

// Eight waves: with four the passes over long lists take longer, with sixteen
// the barriers (39 us for both kernels against 42 and 41, 3 requests of 100k to
// 400k tokens).
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kParts = 2048;          // of a histogram
constexpr int kMaxHeld = 14336;       // blocks whose ends LDS holds, a multiple of 4
constexpr int kMaxOpen = 1024;        // undecided blocks computed in LDS
constexpr int kMaxMarked = 65536;     // blocks with a mark in LDS

struct TopShared {
  int hist[2][kParts];
  uint32_t chosen[kMaxMarked / 32];
  unsigned long long key[kMaxOpen];
  int block[kMaxOpen];
  int tiles[kMaxHeld / kTileBlocks];
  unsigned long long lo[kWaves], hi[kWaves];
  int n[kWaves], f[kWaves];
  int part, above, in, open;
};

// Narrows [lo, hi] around the left-th largest of the keys in it, which
// for_each(f) hands to f one after the other.  Returns the cut: keys from it
// on are wanted, and of those equal to it the first *ties.  Both histograms
// are clear on entry.  A round leaves at most 2^-11 of the range, so there are
// at most six.
template <class K, class ForEach>
__device__ K narrow(TopShared& sh, K lo, K hi, int left, ForEach for_each, int* ties) {
  constexpr int kPer = kParts / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int round = 0;; ++round) {
    const unsigned long long span = (unsigned long long)(hi - lo);
    const int bits = span == 0 ? 0 : 64 - __clzll((long long)span);
    const int shift = max(bits - 11, 0);
    int* hist = sh.hist[round & 1];
    for_each([&](K k) {
      if (k >= lo && k <= hi) atomicAdd(&hist[(int)((k - lo) >> shift)], 1);
    });
    __syncthreads();
    // Counts from the top: each thread kPer parts, then over the waves.
    const int top = kParts - 1 - kPer * tid;
    int c[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = hist[top - i];
      hist[top - i] = 0;  // for the round after next
      mine += c[i];
    }
    const int inc = wave_scan(mine);
    if (lane == 63) sh.n[wave] = inc;
    if (tid == 0) {  // ends the search should the part below not be found
      sh.part = sh.above = 0;
      sh.in = left;
    }
    __syncthreads();
    int above = inc - mine;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (w < wave) above += sh.n[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < left && left <= above + c[i]) {
        sh.part = top - i;
        sh.above = above;
        sh.in = c[i];
      }
      above += c[i];
    }
    __syncthreads();
    left -= sh.above;
    lo += (K)((K)sh.part << shift);
    if (shift == 0 || sh.in == left) {
      *ties = sh.in == left ? 0x7fffffff : left;
      return lo;
    }
    hi = min(hi, (K)(lo + (K)(((K)1 << shift) - 1)));
  }
}

// Lanes that work on a block's 64-bit score: 16 a query head, and four heads at
// a time where the group has them.
__device__ __forceinline__ int exact_lanes(int G) { return G >= 4 ? 64 : 16; }

// 64-bit score of a block, in all of the exact_lanes(G) lanes that work on it;
// l is the number of the lane among them.  What two heads of a lane need is
// asked for together.
__device__ __forceinline__ double exact_score(const SelectArgs& a, int b, int h, int page, int l) {
  typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
  const int G = a.Hq / a.H;
  const int step = exact_lanes(G) / 16;
  const __bf16* lo = a.bounds + ((size_t)page * a.H + h) * 2 * a.D;
  const __bf16* q = a.q + ((size_t)b * a.Hq + h * G) * a.D;
  double best = -__builtin_huge_val();
  for (int g = l / 16; g < G; g += 2 * step) {
    const __bf16 *q0 = q + (size_t)g * a.D, *q1 = q + (size_t)min(g + step, G - 1) * a.D;
    double s0 = 0, s1 = 0;
    for (int d = 4 * (l & 15); d < a.D; d += 64) {
      const bf16x4 lv = *(const bf16x4*)(lo + d), hv = *(const bf16x4*)(lo + a.D + d),
                   v0 = *(const bf16x4*)(q0 + d), v1 = *(const bf16x4*)(q1 + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double x0 = (double)(float)v0[i], x1 = (double)(float)v1[i];
        s0 += (double)(x0 > 0 ? (float)hv[i] : (float)lv[i]) * x0;
        s1 += (double)(x1 > 0 ? (float)hv[i] : (float)lv[i]) * x1;
      }
    }
    // quad_perm 1 0 3 2, 2 3 0 1, row_half_mirror, row_mirror
    s0 += dpp_or_0<0xB1>(s0), s1 += dpp_or_0<0xB1>(s1);
    s0 += dpp_or_0<0x4E>(s0), s1 += dpp_or_0<0x4E>(s1);
    s0 += dpp_or_0<0x141>(s0), s1 += dpp_or_0<0x141>(s1);
    s0 += dpp_or_0<0x140>(s0), s1 += dpp_or_0<0x140>(s1);
    if (s0 > best) best = s0;  // a NaN does not count
    if (s1 > best) best = s1;
  }
  if (step == 4) {
    best = fmax(best, __shfl_xor(best, 16));
    best = fmax(best, __shfl_xor(best, 32));
  }
  return best;
}

}  // namespace

// Workgroup (h, b): the `keep` blocks with the highest scores, the lower index
// first among equals, in index order.  A pass over 12,500 blocks is bound by
// the instructions of its one CU, hence ready-made keys, four to a read.
__global__ __launch_bounds__(kThreads) void select_top_kernel(SelectArgs a, int held) {
  __shared__ TopShared sh;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  uint32_t *kept_lower = (uint32_t*)lds, *kept_upper = kept_lower + held;  // of the first blocks
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = blocks_of(a, b);
  const int32_t* table = a.table + (size_t)b * a.max_blocks;
  unsigned long long* scratch = a.scratch + ((size_t)b * a.H + h) * select_stride(a.max_blocks);
  const Ends* ends = (const Ends*)scratch;
  int32_t* sel = a.sel + ((size_t)b * a.H + h) * a.keep;
  const uint64_t below = (1ull << lane) - 1;

  for (int i = tid; i < 2 * kParts; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.open = 0;
  auto umin = [](uint32_t x, uint32_t y) { return min(x, y); };
  auto umax = [](uint32_t x, uint32_t y) { return max(x, y); };

  // Four blocks from j on (a multiple of 4); zeros behind the last.
  auto fetch4 = [&](int j, u32x4* l, u32x4* u) {
    const u32x4 e0 = load16(ends + j), e1 = load16(ends + j + 2);
    *l = u32x4{e0[0], e0[2], e1[0], e1[2]};
    *u = u32x4{e0[1], e0[3], e1[1], e1[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i >= n) (*l)[i] = (*u)[i] = 0;
  };
  auto lower4 = [&](int j) {
    u32x4 l, u;
    if (j < held) l = *(const u32x4*)(kept_lower + j);
    else fetch4(j, &l, &u);
    return l;
  };
  auto upper4 = [&](int j) {
    u32x4 l, u;
    if (j < held) u = *(const u32x4*)(kept_upper + j);
    else fetch4(j, &l, &u);
    return u;
  };

  // Long lists: as many tiles as blocks are wanted have a block whose lower end
  // is at least the wanted-th largest of the tiles' maxima, so only the tiles
  // that reach that with an upper end, and those with blocks that are always
  // in, need looking at.
  int m = n;
  bool picked = false;
  const int tiles = ceil_div(n, kTileBlocks);
  if (tiles > 4 * (long long)a.keep) {
    const Ends* tops = (const Ends*)a.scratch + select_tiles_at(a.B, a.H, a.max_blocks) +
                       ((size_t)b * a.H + h) * ceil_div(a.max_blocks, kTileBlocks);
    const int front = min(a.first, n), behind = max(n - a.last, front);
    uint32_t lo = ~0u, hi = 0;
    int filled = 0, forced = 0;
    for (int j = tid; j < front; j += kThreads) forced += ends[j].lower == ~0u;
    for (int j = behind + tid; j < n; j += kThreads) forced += ends[j].lower == ~0u;
    for (int t = tid; t < tiles; t += kThreads) {
      const uint32_t k = tops[t].lower;
      filled += k != 0;
      lo = min(lo, k - 1);
      hi = max(hi, k);
    }
    lo = wave_reduce(lo, umin);
    hi = wave_reduce(hi, umax);
    filled = read_lane(wave_scan(filled), 63);
    forced = read_lane(wave_scan(forced), 63);
    if (lane == 0) {
      sh.lo[wave] = lo;
      sh.hi[wave] = hi;
      sh.n[wave] = filled;
      sh.f[wave] = forced;
    }
    __syncthreads();
    filled = forced = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      lo = min(lo, (uint32_t)sh.lo[w]);
      hi = max(hi, (uint32_t)sh.hi[w]);
      filled += sh.n[w];
      forced += sh.f[w];
    }
    __syncthreads();
    const int left = a.keep - forced;
    if (left > 0 && filled > left) {
      int ties;
      const uint32_t reach = narrow<uint32_t>(sh, lo + 1, hi, left, [&](auto f) {
#pragma unroll 1
        for (int t = tid; t < tiles; t += kThreads) f(tops[t].lower);
      }, &ties);
      const int run = ceil_div(ceil_div(tiles, kWaves), 64) * 64;
      const int first = wave * run, last = min(first + run, tiles);
      auto wanted = [&](int t) {
        return t < last && (tops[t].upper >= reach || t * kTileBlocks < front ||
                            (t + 1) * kTileBlocks > behind);
      };
      int mine = 0;
#pragma unroll 1
      for (int t = first; t < last; t += 64) mine += __popcll(__ballot(wanted(t + lane)));
      __syncthreads();
      if (lane == 0) sh.f[wave] = mine;
      __syncthreads();
      int at = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += sh.f[w];
        all += sh.f[w];
      }
      picked = all * (long long)kTileBlocks <= held;
      if (picked) {
        m = all * kTileBlocks;
#pragma unroll 1
        for (int t = first; t < last; t += 64) {
          const uint64_t yes = __ballot(wanted(t + lane));
          if ((yes >> lane) & 1) sh.tiles[at + __popcll(yes & below)] = t + lane;
          at += __popcll(yes);
        }
      }
      __syncthreads();
    }
  }
  // Block that the i-th one looked at is.
  auto block_of = [&](int i) {
    return picked ? sh.tiles[i / kTileBlocks] * kTileBlocks + i % kTileBlocks : i;
  };

  uint32_t lo = ~0u, hi = 0;
  int there = 0, forced = 0;
  for (int j = 4 * tid; j < m; j += 4 * kThreads) {
    u32x4 l, u;
    fetch4(block_of(j), &l, &u);
    if (j < held) {
      *(u32x4*)(kept_lower + j) = l;
      *(u32x4*)(kept_upper + j) = u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      there += l[i] != 0;
      forced += l[i] == ~0u;
      lo = min(lo, l[i] - 1);      // 0 counts as the highest
      hi = max(hi, l[i] + 1);      // ~0 counts as the lowest
    }
  }
  lo = wave_reduce(lo, umin);
  hi = wave_reduce(hi, umax);
  there = read_lane(wave_scan(there), 63);
  forced = read_lane(wave_scan(forced), 63);
  if (lane == 0) {
    sh.lo[wave] = lo;
    sh.hi[wave] = hi;
    sh.n[wave] = there;
    sh.f[wave] = forced;
  }
  __syncthreads();
  there = forced = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    lo = min(lo, (uint32_t)sh.lo[w]);
    hi = max(hi, (uint32_t)sh.hi[w]);
    there += sh.n[w];
    forced += sh.f[w];
  }

  lo += 1;
  hi -= 1;

  // `reach`: lower ends from it on are the highest ones.  The blocks that may
  // be wanted reach it with their upper end; those among them that do not with
  // their lower one reach up to `rival`, and blocks that lie above that, from
  // `sure` on, are in.  The others are undecided.
  const int left = min(a.keep, there) - forced;
  uint32_t sure = 1, reach = 0, rival = 0;
  if (left <= 0) {
    sure = ~0u;  // the forced blocks fill the list
  } else if (there > a.keep) {
    int ties;
    __syncthreads();
    reach = narrow<uint32_t>(sh, lo, hi, left, [&](auto f) {
#pragma unroll 1
      for (int j = 4 * tid; j < m; j += 4 * kThreads) {
        const u32x4 l = lower4(j);
#pragma unroll
        for (int i = 0; i < 4; ++i) f(l[i]);
      }
    }, &ties);
#pragma unroll 1
    for (int j = 4 * tid; j < m; j += 4 * kThreads) {
      const u32x4 l = lower4(j), u = upper4(j);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (l[i] < reach) rival = max(rival, u[i]);
    }
    rival = wave_reduce(rival, umax);
    if (lane == 0) sh.f[wave] = (int)rival;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) rival = max(rival, (uint32_t)sh.f[w]);
    if (rival < reach) rival = 0;                  // none
    if (ties != 0x7fffffff) rival = ~0u - 1;       // equal lower ends at the cut
    sure = max(reach, rival + 1);
  }
  auto open = [&](uint32_t l, uint32_t u) { return u >= reach && l <= rival; };

  if (rival != 0) {
    // Undecided blocks: listed in LDS, computed in 64 bits, and chosen by
    // counting the better ones.
    const int lanes = exact_lanes(a.Hq / a.H), sub = tid & (lanes - 1);
    int in = 0;
    for (int i = tid; i < min(ceil_div(m, 32), kMaxMarked / 32); i += kThreads) sh.chosen[i] = 0;
#pragma unroll 1
    for (int j = 4 * tid; j < m; j += 4 * kThreads) {
      const u32x4 l = lower4(j), u = upper4(j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        in += l[i] >= sure;
        if (open(l[i], u[i])) {
          const int at = atomicAdd(&sh.open, 1);
          if (at < kMaxOpen) sh.block[at] = j + i;
        }
      }
    }
    in = read_lane(wave_scan(in), 63);
    if (lane == 0) sh.n[wave] = in;
    __syncthreads();
    const int opened = sh.open;
    if (opened > kMaxOpen || m > kMaxMarked) {
      // Too many (equal scores, very long lists): 64-bit keys of all that may
      // be wanted in place of the intervals, and the same narrowing on them.
#pragma unroll 1
      for (int j = tid / lanes; j < n; j += kThreads / lanes) {
        const Ends v = ends[j];
        unsigned long long k = v.lower == ~0u ? kForced : kMissing;
        if (v.lower != ~0u && v.upper >= reach) k = order_key(exact_score(a, b, h, table[j], sub));
        // A block's lanes run together: all have read v before one writes.
        if (sub == 0) scratch[j] = k;
      }
      __syncthreads();
      unsigned long long klo = ~0ull, khi = 0;
      for (int j = tid; j < n; j += kThreads) {
        const unsigned long long k = scratch[j];
        if (k != kMissing && k != kForced) {
          klo = min(klo, k);
          khi = max(khi, k);
        }
      }
#pragma unroll 1
      for (int o = 32; o > 0; o >>= 1) {
        klo = min(klo, (unsigned long long)__shfl_xor((long long)klo, o));
        khi = max(khi, (unsigned long long)__shfl_xor((long long)khi, o));
      }
      if (lane == 0) {
        sh.lo[wave] = klo;
        sh.hi[wave] = khi;
      }
      for (int i = tid; i < 2 * kParts; i += kThreads) (&sh.hist[0][0])[i] = 0;
      __syncthreads();
      for (int w = 0; w < kWaves; ++w) {
        klo = min(klo, sh.lo[w]);
        khi = max(khi, sh.hi[w]);
      }
      int ties;
      const unsigned long long cut = narrow<unsigned long long>(sh, klo, khi, left, [&](auto f) {
        for (int j = tid; j < n; j += kThreads) f(scratch[j]);
      }, &ties);
      int out = 0, seen = 0;
      for (int j0 = 0; j0 < n; j0 += kThreads) {
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
        for (int w = 0; w < kWaves; ++w) {
          if (w < wave) {
            r += sh.n[w];
            e += sh.f[w];
          }
          out += sh.n[w];
          seen += sh.f[w];
        }
        const int to = r + min(e, ties);
        if ((k > cut || (k == cut && e < ties)) && to < a.keep) sel[to] = j;
      }
      for (int i = out + min(seen, ties) + tid; i < a.keep; i += kThreads) sel[i] = -1;
      return;
    }
    in = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) in += sh.n[w];
#pragma unroll 1
    for (int c = tid / lanes; c < opened; c += kThreads / lanes) {
      const double s = exact_score(a, b, h, table[block_of(sh.block[c])], sub);
      if (sub == 0) sh.key[c] = order_key(s);
    }
    __syncthreads();
#pragma unroll 1
    for (int c = tid; c < opened; c += kThreads) {
      const unsigned long long k = sh.key[c];
      const int j = sh.block[c];
      int better = 0;
      for (int i = 0; i < opened; ++i)
        better += sh.key[i] > k || (sh.key[i] == k && sh.block[i] < j);
      if (better < left + forced - in) atomicOr(&sh.chosen[j / 32], 1u << (j & 31));
    }
    __syncthreads();
  }

  // Out in index order: each wave counts its run of blocks, then writes it,
  // four blocks a lane.
  const int run = ceil_div(ceil_div(m, kWaves), 256) * 256;
  const int j0 = wave * run, j1 = min(j0 + run, m);
  auto chosen4 = [&](int j) {
    uint32_t bits = 0;
    if (j < j1) {
      const u32x4 l = lower4(j);
#pragma unroll
      for (int i = 0; i < 4; ++i) bits |= (uint32_t)(l[i] >= sure) << i;
      if (rival != 0) bits |= (sh.chosen[j / 32] >> (j & 31)) & 15;
    }
    return bits;
  };
  int mine = 0;
#pragma unroll 1
  for (int j = j0; j < j1; j += 256) mine += __popc(chosen4(j + 4 * lane));
  mine = read_lane(wave_scan(mine), 63);
  __syncthreads();
  if (lane == 0) sh.f[wave] = mine;
  __syncthreads();
  int at = 0, out = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) at += sh.f[w];
    out += sh.f[w];
  }
#pragma unroll 1
  for (int j = j0; j < j1; j += 256) {
    const uint32_t bits = chosen4(j + 4 * lane);
    const int upto = wave_scan((int)__popc(bits));
    int r = at + upto - __popc(bits);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((bits >> i) & 1 && r < a.keep) sel[r++] = block_of(j + 4 * lane + i);
    at += read_lane(upto, 63);
  }
  for (int i = out + tid; i < a.keep; i += kThreads) sel[i] = -1;
}

namespace {

template <int D, int kHeads>
hipError_t launch_score(const SelectArgs& a, hipStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const hipError_t e = once_per_device(done, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(select_score_kernel<D, kHeads>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, 4 * BoundsTile<D>::kLds);
  });
  if (e != hipSuccess) return e;
  select_score_kernel<D, kHeads><<<BoundsTile<D>::kPerCu * kCus, 256, 4 * BoundsTile<D>::kLds, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_score_heads(const SelectArgs& a, hipStream_t stream) {
  return a.H % 4 == 0   ? launch_score<D, 4>(a, stream)
         : a.H % 2 == 0 ? launch_score<D, 2>(a, stream)
                        : launch_score<D, 1>(a, stream);
}

hipError_t launch_top(const SelectArgs& a, hipStream_t stream) {
  const int held = std::min((a.max_blocks + 3) / 4 * 4, kMaxHeld);
  static std::atomic<unsigned long long> done{0};
  const hipError_t e = once_per_device(done, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(select_top_kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld * 8);
  });
  if (e != hipSuccess) return e;
  select_top_kernel<<<dim3(a.H, a.B), kThreads, held * 8, stream>>>(a, held);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_select(const SelectArgs& a, hipStream_t stream) {
  const hipError_t e = a.D == 64    ? launch_score_heads<64>(a, stream)
                       : a.D == 128 ? launch_score_heads<128>(a, stream)
                       : a.D == 256 ? launch_score_heads<256>(a, stream)
                                    : hipErrorInvalidValue;
  return e == hipSuccess ? launch_top(a, stream) : e;
}

}  // namespace mova

// What the two kernels of the chunk attention share: the rows of a request, the
// line of work over the batch, where results go and how parts of them are joined.
#pragma once

#include "paged.h"

namespace mova {

// Requests of so few rows (tokens times query heads of a key head) are the few-rows
// kernel's, where it is launched: in batches with as few on average, and in those of
// kFewRequests, where some will have few.  (64 requests of 500 to 8000 tokens, 32 heads
// over 8, by that kernel and by the one of many rows: a token each 128 and 157 us, four
// tokens, which fill sixteen rows, 142 and 165; eight, as two times sixteen, 260 and
// 177.  60 with a token and 4 with 512, by both kernels and by one: 221 and 272 us; 32
// with one and 32 with 64: 208 and 228.  Where no request has few rows the launch costs
// 2 to 4 us, and where few short ones have, more: windows over 37 requests 87 and 78.
// Below 32 requests, single tokens after 500 to 8000 and one chunk of 512: 8 requests 99
// by both and 83 by one, 16 112 and 104, 24 118 and 116, 31 157 and 159; after 100 to 1000
// 24 65 and 55; in 8 bits, where a chunk of 2048 pays for the launch, 8 196 and 193, 16 189
// and 202, 24 183 and 209.)
constexpr int kFewRows = 16, kFewRequests = 32;

// What a stretch leaves to be joined.
struct Split {
  long long row0;    // the rows' place in the output
  long long before;  // units of the stretch ahead of them
  int n;             // stretches; 0: nothing was split; -x: in the middle of what the
                     // stretch x before this one left
  int lo, hi;        // keys
  int rows, heads;   // tokens and query heads
  int pad;
};
// Rows whose keys were split over stretches: each stretch leaves its part, at place
// 2 slot + 1 where it holds the beginning and 2 slot where it goes on, and the one that
// they begin in says what there is to join.
struct Parts {
  Split* split;  // [a workgroup]
  float* ml;     // [two a workgroup][rows][2] maximum (in powers of two) and sum
  float* o;      // [two a workgroup][rows][D] out, divided by the sum
};

constexpr size_t split_floats(int groups) { return (size_t)groups * sizeof(Split) / 4; }
static_assert(sizeof(Split) % 8 == 0, "whole words");

// Of the few-rows kernel, for calls of T tokens in B requests of at most `most` keys:
// workgroups, key heads (tracks) of one, floats of scratch, the parts in the scratch, and
// the launch, without the joining of its parts.
int chunk_few_groups(int T, int B, int H, int D, long long most);
int chunk_few_tracks(int H);
size_t chunk_few_floats(int groups, int H, int D);
Parts chunk_few_parts(float* scratch, int groups, int H);
hipError_t launch_chunk_few(const ChunkArgs& a, const Parts& parts, int groups, hipStream_t stream);

// Workgroups for a line of at most `units` units of work, in stretches of `least` or more:
// as many as there can be stretches (neighbours are dealt out in eights), up to `most`.
inline int groups_for(double units, int least, int most) {
  return units >= (double)least * most ? most : ((int)(units / least) / 8 + 1) * 8;
}

namespace {

constexpr int kCus = 256;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// The lane's number, formed anew: nothing that follows from it is held from before.
__device__ __forceinline__ int lane_anew() {
  uint32_t all = ~0u;
  asm volatile("" : "+s"(all));
  int lane = (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0u));
  asm volatile("" : "+v"(lane));
  return lane;
}

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

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;

// 8 elements of the pool as bf16 (exact).
template <bool kFp8>
__device__ __forceinline__ Frag16 load8(const void* pool, size_t at) {
  Frag16 f;
  if constexpr (kFp8) {
    const uint2 w = *reinterpret_cast<const uint2*>((const uint8_t*)pool + at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f.h[i] = (__bf16)__builtin_amdgcn_cvt_f32_fp8((int)((i < 4 ? w.x : w.y) >> 8 * (i % 4)), 0);
  } else {
    f.u = load16((const bf16_t*)pool + at);
  }
  return f;
}
// One element's bits as bf16.
template <bool kFp8>
__device__ __forceinline__ uint32_t load1(const void* pool, size_t at) {
  if constexpr (kFp8)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)pool)[at], 0)) >> 16;
  else
    return ((const uint16_t*)pool)[at];
}

struct Shared {
  long long tmp[8];
  long long first;
  int b;
};
// As line_begin, for workgroups of kWaves waves.  `slot`: which stretch; `least`: units of
// one at least.
template <int kWaves, class Cost>
__device__ __forceinline__ bool chunk_line(int B, int slot, int slots, int least, Cost cost,
                                           Shared& sh, Line* line) {
  constexpr int kThreads = 64 * kWaves;
  const int per = ceil_div(B, kThreads);
  const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
  // The thread's first request (up to 256 the only one) is looked at once.
  const long long cost0 = b0 < b1 ? cost(b0) : 0;
  auto cost_of = [&](int b) { return b == b0 ? cost0 : cost(b); };
  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += cost_of(b);
  long long before = block_exclusive_scan<kWaves>(mine, sh.tmp, &total);
  line->stretch = max(floor_div(total + slots - 1, slots), (long long)least);
  line->start = line->stretch * slot;
  line->end = min(line->start + line->stretch, total);
  if (before <= line->start && line->start < before + mine) {
    long long at = before;
    int b = b0;
    for (long long c; line->start >= at + (c = cost_of(b)); ++b) at += c;
    sh.b = b;
    sh.first = at;
  }
  __syncthreads();
  if (line->start >= total) return false;
  line->b = __builtin_amdgcn_readfirstlane(sh.b);
  line->first = (long long)read_lane((double)sh.first, 0);
  return true;
}

// Where a row's result goes: its place in the output, or in the parts.
template <int D>
struct Sink {
  bf16_t* out;  // null: the parts
  float* lse;   // null: none
  float* o;
  float* ml;
  __device__ __forceinline__ void put1(int c, float y) const {
    if (out != nullptr) out[c] = (bf16_t)y;
    else o[c] = y;
  }
  // m: the maximum in powers of two, l: the sum of exp2(. - m).
  __device__ __forceinline__ void put_sum(float m, float l) const {
    if (out == nullptr) {
      ml[0] = m;
      ml[1] = l;
    } else if (lse != nullptr) {
      *lse = l == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
    }
  }
};

// Rows whose sums the matrix products left infinite or NaN, formed again by one wave,
// up to 32 side by side: o = sum_p exp2(s_p - base) v_p over keys [lo, hi), for channels
// [32 c0, 32 c1).  A lane has a row (lanes i and i + 32 the same): its query q (null:
// none), the positions [lower, limit] that it sees and its base; put(c, y) takes factor
// times its channels one by one.
//
// Finite values are summed as ever, with weights to 2^-16; where such a sum passes the
// largest number, it is formed once more with weights 2^-40 as large.  Values that are
// infinite or NaN take part as zeros, and which of them a row has is counted by a product
// of their kinds with the kinds of the weights: so nothing shows of a value that a row
// does not see, and one with a weight makes its channel infinite, or NaN.
//
// Keys and values come straight from the pool, and the logits are formed again for each
// 32 channels, which keeps this in the registers that the kernels have.  Bound by round
// trips to memory, some 3 to 5 us for 32 keys, 32 rows and 32 channels; a row at a time, with
// its values key by key, took 140 times a call where this takes 8.  (A value that all rows
// of a prompt see, 32 heads over 8 of 128: 512 tokens 294 us, a row at a time 5169, without
// the value 47; 2048 tokens 657, 12,358 and 86; 8192 tokens 9.7 ms, without it 0.58.)
template <int D, bool kFp8, class Put>
__device__ __forceinline__ void attend_again(const ChunkArgs& a, FastDiv by_block, int b, int h,
                                             const bf16_t* q, float qs, float base, int limit,
                                             int lower, int lo, int hi, int c0, int c1,
                                             float factor, Put put) {
  constexpr float kDown = 0x1p-40f;
  const int lane = lane_anew(), r32 = lane & 31, half = lane >> 5;
  const int32_t* table = a.table + (size_t)b * a.max_blocks;
  const size_t row = (size_t)a.H * D;  // elements between keys
  auto slot_of = [&](int p) {
    if (p >= hi) return -1;
    const int j = fast_div(p, by_block), page = table[j];
    if (page < 0 || page >= a.num_blocks) return -1;
    return page * a.block_size + (p - j * a.block_size);
  };
  union Eight {
    uint16_t e[8];
    bf16x8 h;
  };
  // Twice for each 32 channels at most: with weights as they are, and smaller.
  uint32_t over = 0;               // a bit a channel of the lane: the first sum was too large
  uint32_t plus = 0, minus = 0;    // infinities of its values; both: NaN
#pragma unroll 1
  for (int turn = 2 * c0; turn < 2 * c1; ++turn) {
    const int c = turn >> 1;
    const bool again = turn & 1;
    if (again && !__any(over != 0)) continue;
    if (!again) plus = minus = 0;
    const size_t channel = (size_t)h * D + 32 * c + r32;  // that the lane reads
    f32x16 o;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    int next = slot_of(lo + r32);
#pragma unroll 1
    for (int p0 = lo; p0 < hi; p0 += 32) {
      const int slot = next;
      next = slot_of(p0 + 32 + r32);
      const uint32_t present = (uint32_t)__ballot(slot >= 0);
      if (present == 0) continue;
      // The lane's logits and values are of keys 8 (i / 4) + 4 half + i % 4.
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = __builtin_amdgcn_ds_bpermute(4 * (8 * (i / 4) + 4 * half + i % 4), slot);
        v[i] = load1<kFp8>(a.v_cache, (size_t)(uint32_t)max(key, 0) * row + channel);
        if (key < 0) v[i] = 0u;
      }
      f32x16 s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
      const size_t at = (size_t)(uint32_t)max(slot, 0) * row + (size_t)h * D + 8 * half;
#pragma unroll 4
      for (int u = 0; u < D / 16; ++u) {
        Frag16 x;
        x.u = u32x4{0u, 0u, 0u, 0u};
        if (q != nullptr) x.u = load16(q + 16 * u + 8 * half);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(load8<kFp8>(a.k_cache, at + 16 * u).h, x.h, s, 0,
                                                    0, 0);
      }
      // Bits of the keys that the row sees; the lane's begin at 4 half.
      const int above = limit - p0, below = lower - p0;
      uint32_t seen = above < 0 ? 0u : present;
      if (above < 31) seen &= (2u << max(above, 0)) - 1;
      if (below > 0) seen &= below > 31 ? 0u : ~0u << below;
      seen >>= 4 * half;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float w[8];
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          odd = odd || (v[8 * y + e] & 0x7f80u) == 0x7f80u;
          const bool sees = (seen >> (16 * y + 8 * (e / 4) + e % 4)) & 1;
          w[e] = sees ? __builtin_amdgcn_exp2f(fmaf(s[8 * y + e], qs, -base)) : 0.f;
        }
        Eight high, low, value;
        if (__any(odd)) {
          // A value's kind: 1 for one that adds to plus infinity, 64 to minus, 65 NaN.  A
          // weight's: 1, or 4096 where it is rounded to 0 (times an infinity NaN).
          // Sums of 16 keys stay below 2^24.
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t bits = v[8 * y + e];
            const bool inf = (bits & 0x7fffu) == 0x7f80u, nan = (bits & 0x7fffu) > 0x7f80u;
            const bool sees = (seen >> (16 * y + 8 * (e / 4) + e % 4)) & 1;
            value.e[e] = f32_to_bf16_bits(nan ? 65.f : inf ? (bits >> 15 ? 64.f : 1.f) : 0.f);
            high.e[e] = f32_to_bf16_bits(w[e] > 0.f ? 1.f : sees ? 4096.f : 0.f);
            if (inf || nan) v[8 * y + e] = 0u;
          }
          f32x16 sum;
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[i] = 0.f;
          sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value.h, high.h, sum, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t n = (uint32_t)sum[i];
            const bool none = n >> 12 != 0;  // of a weight of 0
            plus |= (uint32_t)(none || (n & 63u) != 0) << i;
            minus |= (uint32_t)(none || (n >> 6 & 63u) != 0) << i;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = again ? w[e] * kDown : w[e];
          high.e[e] = f32_to_bf16_bits(x);
          low.e[e] = f32_to_bf16_bits(x - __builtin_bit_cast(float, (uint32_t)high.e[e] << 16));
          value.e[e] = (uint16_t)v[8 * y + e];
        }
        o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value.h, high.h, o, 0, 0, 0);
        o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value.h, low.h, o, 0, 0, 0);
      }
    }
    if (!again) over = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool up = (plus >> i) & 1, dn = (minus >> i) & 1, fits = fabsf(o[i]) < __builtin_huge_valf();
      if (!again) over |= (uint32_t)(!up && !dn && !fits) << i;
      float y = o[i] * factor;
      if (again) y *= 1 / kDown;
      if (up || dn) y = (up ? __builtin_huge_valf() : 0.f) - (dn ? __builtin_huge_valf() : 0.f);
      if (!again || ((over >> i) & 1)) put(32 * c + 8 * (i / 4) + 4 * half + i % 4, y);
    }
  }
}

// Zeros for the rows that have no token in the cache; the whole grid takes part.
__device__ __forceinline__ void clear_rows(const ChunkArgs& a, int tid) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const Chunk c = chunk_of(a, b);
    const size_t from = (size_t)(c.row0 + c.live) * a.Hq, to = (size_t)(c.row0 + c.rows) * a.Hq;
    for (size_t i = from * a.D + tid * 8; i < to * a.D; i += blockDim.x * 8)
      store16(a.out + i, u32x4{0u, 0u, 0u, 0u});
    if (a.lse != nullptr)
      for (size_t i = from + tid; i < to; i += blockDim.x) a.lse[i] = -__builtin_huge_valf();
  }
}

// Four channels of a joined row, and its lse once a row.
template <int D>
__device__ __forceinline__ void put_joined(const ChunkArgs& a, size_t row, int channel, f32x4 o,
                                           float m, float sum) {
  uint2 y;
  y.x = (uint32_t)f32_to_bf16_bits(o[0]) | ((uint32_t)f32_to_bf16_bits(o[1]) << 16);
  y.y = (uint32_t)f32_to_bf16_bits(o[2]) | ((uint32_t)f32_to_bf16_bits(o[3]) << 16);
  *reinterpret_cast<uint2*>(a.out + row * D + channel) = y;
  if (a.lse != nullptr && channel == 0)
    a.lse[row] = sum == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}
__device__ __forceinline__ float finite_or_0(float m) {
  return m == -__builtin_huge_valf() ? 0.f : m;
}
typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;

// A record as the whole wave has it: what is found from it takes scalar registers, and no
// branches per lane.
__device__ __forceinline__ Split split_of(const Split* from) {
  union {
    Split s;
    int w[sizeof(Split) / 4];
  } x;
  x.s = *from;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Split) / 4); ++i) x.w[i] = __builtin_amdgcn_readfirstlane(x.w[i]);
  return x.s;
}

// o += w y; what a part without weight holds may be anything.
__device__ __forceinline__ void add_part(f32x4& o, float w, const f32x4& y) {
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = w == 0.f ? o[c] : fmaf(w, y[c], o[c]);
}

// Joins share `share` of `shares` of the parts of `rows` rows, n of each, with kWaves
// waves.  part_of(r, i) is a part's place, or -1; row_of(r) the row's
// in the output, or -1.
//
// Of up to kFew parts a row has D / 4 lanes, and a wave asks for all parts of kSets such
// sets of rows at once: there are many rows, and what they cost is the round trips.  (The
// parts of 255 tiles of 256 rows, 128 wide, two of each: a wave a row 44 us, so 20; 28
// with a branch around each read.)  Of more parts a row has a wave: the maxima and sums
// come first, a lane a part, and then the parts, 64 / (D / 4) times eight of them at
// once.  (24 parts of 32 rows: 30 us with a branch around each read, 8 so.)
template <int D, int kWaves, int kFew, int kSets, class PartOf, class RowOf>
__device__ __forceinline__ void join_rows(const ChunkArgs& a, const Parts& parts, int rows, int n,
                                          int share, int shares, PartOf part_of, RowOf row_of) {
  constexpr int kLanes = D / 4, kAtOnce = 64 / kLanes, kBatch = 8;
  const int lane = threadIdx.x & 63;
  const int wave = share * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = shares * kWaves;
  const int mine = lane / kLanes, channel = lane % kLanes * 4;
  if (n <= kFew) {
    for (int r0 = wave * kAtOnce + mine; r0 < rows; r0 += waves * kAtOnce * kSets) {
      float pm[kSets][kFew], pl[kSets][kFew];
      uint32_t there[kSets];  // a bit a part
      f32x4 y[kSets][kFew];
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        const int r = r0 + s * waves * kAtOnce;
        const bool live = r < rows && row_of(r) >= 0;
        there[s] = 0;
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
          // (Reads of the first part where there is none: a branch would wait for the
          // loads before it.)
          const long long p = live && i < n ? part_of(r, i) : -1, at = max(p, 0ll);
          there[s] |= (uint32_t)(p >= 0) << i;
          pm[s][i] = parts.ml[2 * at];
          pl[s][i] = parts.ml[2 * at + 1];
          y[s][i] = *reinterpret_cast<const f32x4*>(parts.o + (size_t)at * D + channel);
        }
      }
#pragma unroll
      for (int s = 0; s < kSets; ++s)
#pragma unroll
        for (int i = 0; i < kFew; ++i)
          if (!(there[s] >> i & 1)) pl[s][i] = 0.f;
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        const int r = r0 + s * waves * kAtOnce;
        const long long row = r < rows ? row_of(r) : -1;
        if (row < 0) continue;
        float m = -__builtin_huge_valf(), sum = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kFew; ++i)
          if (pl[s][i] != 0.f) m = fmaxf(m, pm[s][i]);
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
          pl[s][i] = pl[s][i] == 0.f
                         ? 0.f
                         : pl[s][i] * __builtin_amdgcn_exp2f(pm[s][i] - finite_or_0(m));
          sum += pl[s][i];
        }
        const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < kFew; ++i) add_part(o, pl[s][i] * f, y[s][i]);
        put_joined<D>(a, (size_t)row, channel, o, m, sum);
      }
    }
    return;
  }
  for (int r = wave; r < rows; r += waves) {
    const long long row = row_of(r);
    if (row < 0) continue;
    float m = -__builtin_huge_valf(), sum = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    // A lane's part among those from x0 on: its maximum and sum.
    auto of_lane = [&](int x0) {
      const long long p = x0 + lane < n ? part_of(r, x0 + lane) : -1, at = max(p, 0ll);
      f32x2 x = {parts.ml[2 * at], parts.ml[2 * at + 1]};
      if (p < 0) x[1] = 0.f;
      return x;
    };
    const f32x2 first = of_lane(0);  // held: n is mostly below 64
    if (first[1] != 0.f) m = first[0];
    for (int x0 = 64; x0 < n; x0 += 64) {
      const f32x2 x = of_lane(x0);
      if (x[1] != 0.f) m = fmaxf(m, x[0]);
    }
    m = wave_reduce(m, [](float x, float y) { return fmaxf(x, y); });
    auto weight = [&](int x0) {
      f32x2 x = first;
      if (x0 > 0) x = of_lane(x0);
      return x[1] == 0.f ? 0.f : x[1] * __builtin_amdgcn_exp2f(x[0] - finite_or_0(m));
    };
    for (int x0 = 0; x0 < n; x0 += 64) sum += weight(x0);
    sum = wave_sum(sum);
    const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
    for (int x0 = 0; x0 < n; x0 += 64) {
      const float w = weight(x0) * f;
#pragma unroll 1
      for (int x = 0; x < min(n - x0, 64); x += kAtOnce * kBatch) {
        f32x4 y[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = min(x0 + x + i * kAtOnce + mine, n - 1);
          y[i] = *reinterpret_cast<const f32x4*>(parts.o + (size_t)max(part_of(r, at), 0ll) * D +
                                                 channel);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) add_part(o, __shfl(w, x + i * kAtOnce + mine), y[i]);
      }
    }
#pragma unroll
    for (int step = kLanes; step < 64; step *= 2)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] += __shfl_xor(o[c], step);
    if (mine == 0) put_joined<D>(a, (size_t)row, channel, o, m, sum);
  }
}

}  // namespace

}  // namespace mova

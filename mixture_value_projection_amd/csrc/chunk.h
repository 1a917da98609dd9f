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
// 2 to 4 us, and where few short ones have, more: windows over 37 requests 87 and 78.)
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

// Of the few-rows kernel: floats of scratch, workgroups, key heads (tracks) of one, the
// parts in the scratch, and the launch, without the joining of its parts.
size_t chunk_few_scratch_floats(int D);
int chunk_few_groups(const ChunkArgs& a);
int chunk_few_tracks(int H);
Parts chunk_few_parts(float* scratch);
hipError_t launch_chunk_few(const ChunkArgs& a, const Parts& parts, hipStream_t stream);

namespace {

constexpr int kCus = 256;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// The lane's number, formed anew: nothing that follows from it is held from before.
__device__ __forceinline__ int lane_anew() {
  int lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
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

// One row by one wave with everything in fp32, a lane a key for the logits and
// D / 64 channels a lane for the values: the maximum first, then weights and
// sums.  Only keys that take part are touched, so infinite and NaN values of
// others do not show, and sums that pass the largest number are formed with
// weights 2^-32 as large (a row has at most 2^30 keys).  For the rows whose sums
// the matrix products left infinite or NaN.
template <int D, bool kFp8>
__device__ __forceinline__ void attend_row(const ChunkArgs& a, FastDiv by_block, int b, int h,
                                           const bf16_t* q, int lo, int hi, const Sink<D>& sink) {
  constexpr int kPer = D / 64;
  constexpr float kDown = 0x1p-32f;
  const int lane = lane_anew();
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
#pragma unroll 1
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
  float l = 0.f, o[kPer] = {}, less[kPer] = {};
#pragma unroll 1
  for (int p = lo; p < hi; p += 64) {
    const long long at = place(p + lane);
    const float w = at >= 0 ? __builtin_amdgcn_exp2f(logit(at) - safe) : 0.f;
    l += w;
#pragma unroll 1
    for (uint64_t there = __ballot(at >= 0); there != 0; there &= there - 1) {
      const int i = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)there) - 1);
      const float wi = __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, w), i));
      const uint32_t low = (uint32_t)read_lane((int)at, i), high = (uint32_t)read_lane((int)(at >> 32), i);
      const size_t from = ((size_t)high << 32 | low) + lane * kPer;
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
    sink.put1(lane * kPer + j, l == 0.f ? 0.f : y);
  }
  if (lane == 0) sink.put_sum(m, l);
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

// Attention of a chunk of new tokens per request over the paged key-value cache
// that already holds them (prompts, chunks of prompts, drafts).
//
//   out_ti = sum_p exp(s_tip - m_ti) v_p / sum_p exp(s_tip - m_ti),  s_tip = scale q_ti . k_p
//
// over the positions p up to the token's own, in one pass over the keys with the
// running maximum m and sum of a softmax.
#include <algorithm>
#include <atomic>

#include "chunk.h"
#include "kernels.h"

namespace mova {

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

template <int D, bool kFp8>
struct Tile {
  static constexpr int kWaves = 8, kThreads = 64 * kWaves;
  // Waves that share 32 rows and have a part of the channels each: of 256, the sums
  // and what else a wave holds would not fit its registers.  (The products with the
  // keys are then formed twice.)
  static constexpr int kSplit = D == 256 ? 2 : 1;
  static constexpr int kRowWaves = kWaves / kSplit;
  static constexpr int kRows = 32 * kRowWaves;         // rows (token and query head) of a workgroup
  static constexpr int kKeys = D == 256 ? 32 : 64;     // of a tile
  static constexpr int kParts = kKeys / 32;
  static constexpr bool kQueriesInLds = D == 256;
  // Bytes between rows in LDS: padded so that the 8 rows of a phase of the keys'
  // reads, and the 4 that 16 lanes of a transposing read take, lie in different
  // banks, with all of a tile's places at constant offsets from one address.
  static constexpr int kKeyRow = 2 * D + 16;
  static constexpr int kValueRow = 2 * D + 32;
  static constexpr int kValuesAt = kKeys * kKeyRow;    // in a stage, behind the keys
  static constexpr int kStage = kValuesAt + kKeys * kValueRow;
  static constexpr int kQueries = kQueriesInLds ? kRows * kKeyRow : 0;
  static constexpr int kSlots = 8;                     // tiles whose keys' slots are at hand
  static constexpr int kLds = kQueries + 2 * kStage + kSlots * kKeys * 4;
  // Staging: a thread moves kLoads 16-byte pieces of the pool a side.
  static constexpr int kPieces = D * (kFp8 ? 1 : 2) / 16;  // of a key
  static constexpr int kTotal = kKeys * kPieces;
  static constexpr int kLoads = (kTotal + kThreads - 1) / kThreads;
  static constexpr int kStep = kThreads / kPieces;         // keys between a thread's pieces
  // 8-bit values are multiplied as fp16, with weights up to 2^kLift rather than 1
  // so that the small ones keep their bits.
  static constexpr float kLift = kFp8 ? 14.f : 0.f;
  // Sums are brought to a new maximum once it is this much higher (in powers of two).
  static constexpr float kSlack = kFp8 ? 1.f : 8.f;
};

// How the rows of a request and key head are cut: blocks of `tokens` tokens with
// `heads` of the query heads.
struct Cut {
  int tokens, heads, head_blocks;
};
Cut cut_of(int G, int rows) {
  Cut c;
  c.head_blocks = ceil_div(G, rows);
  c.heads = ceil_div(G, c.head_blocks);
  c.tokens = std::max(1, rows / c.heads);
  return c;
}

// What a request brings to the line of work, in keys: each of its row tiles reads
// keys [lo, hi), and kFixed more for what a tile costs beside them.  (Of 0, 320 and 640:
// a prompt of 8192 tokens 697, 596 and 599 us, 24 requests of 8 bits 606, 539 and 542,
// 200 of 40 tokens 174, 113 and 127.)
constexpr int kFixed = 320;
// A stretch of the line is at least this long.  (Of 256, 512 and 1024: 19 tokens after
// 130 18.6, 16.9 and 25.0 us, 64 after 2000 36, 42 and 49, 32 after 8000 60, 39 and 41, 4
// requests of 64 after 500 31, 33 and 47, a prompt of 512 39, 38 and 46.)
constexpr int kLeastStretch = 512;
struct Load {
  int at, live, tokens, window;
  __device__ __forceinline__ int tiles() const { return ceil_div(live, tokens); }
  __device__ __forceinline__ int hi(int k) const {
    return at + min(live, (int)min((long long)(k + 1) * tokens, (long long)live));
  }
  __device__ __forceinline__ int lo(int k) const {
    return window > 0 ? max(0, at + k * tokens + 1 - window) : 0;
  }
  __device__ __forceinline__ long long units(int k) const { return hi(k) - lo(k) + kFixed; }
  // Units of tiles 0 .. n - 1.
  __device__ __forceinline__ long long before(int n) const {
    const long long N = n, s = tokens;
    long long sum = N * ((long long)at + kFixed) + s * (N * (N + 1) / 2);
    if (n > 0 && n == tiles()) sum -= N * s - live;
    if (window > 0) {
      const int first = window - 1 - at < 0 ? 0 : (window - 1 - at) / tokens + 1;
      if (first < n) {
        const long long m = n - first;
        sum -= m * ((long long)at + 1 - window) + s * ((long long)(n - 1 + first) * m / 2);
      }
    }
    return sum;
  }
  // The tile that unit x (< before(tiles())) lies in.
  __device__ __forceinline__ int tile_at(long long x) const {
    int lo_ = 0, hi_ = tiles();
    while (hi_ - lo_ > 1) {
      const int mid = (lo_ + hi_) >> 1;
      if (before(mid) <= x) lo_ = mid;
      else hi_ = mid;
    }
    return lo_;
  }
};
// Whether the request is this kernel's.
__device__ __forceinline__ bool many_rows(const ChunkArgs& a, const Chunk& c) {
  return c.live * (a.Hq / a.H) > a.few;
}

// Key tiles [begin, end) that units [x0, x1) of a row tile over keys [lo, hi) stand
// for; all of them together are [first, last).
struct Segment {
  int begin, end, first, last;
};
template <int kKeys>
__device__ __forceinline__ Segment segment_of(int lo, int hi, long long x0, long long x1) {
  const long long units = hi - lo + kFixed;
  Segment s;
  s.first = lo / kKeys;
  s.last = ceil_div(hi, kKeys);
  auto at = [&](long long x) {
    if (x <= 0) return s.first;
    if (x >= units) return s.last;
    return (lo + (int)max(x - kFixed, 0ll)) / kKeys;
  };
  s.begin = at(x0);
  s.end = at(x1);
  return s;
}

// Maximum of lanes i and i + 32, in both.
__device__ __forceinline__ float max_of_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

__device__ __forceinline__ float sum_of_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// 16 e4m3 elements as bf16 or fp16 (both exact).
template <bool kHalf>
__device__ __forceinline__ void widen16(const u32x4& w, u32x4* a, u32x4* b) {
  auto two = [](uint32_t x, auto upper) {
    if constexpr (kHalf)
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(
                                              (int)x, 1.f, decltype(upper)::value));
    else
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                              (int)x, 1.f, decltype(upper)::value));
  };
  using std::false_type;
  using std::true_type;
  *a = u32x4{two(w[0], false_type{}), two(w[0], true_type{}), two(w[1], false_type{}),
             two(w[1], true_type{})};
  *b = u32x4{two(w[2], false_type{}), two(w[2], true_type{}), two(w[3], false_type{}),
             two(w[3], true_type{})};
}

}  // namespace

// Rows, tokens times query heads of a key head, are many here, so a key tile is used
// by 256 of them (128 where rows have 256 channels) and the matrix products bound it.
//
// A workgroup has eight waves of 32 rows.  Logits are K Q^T, which leaves 32 rows across
// the lanes and a tile's 64 keys down the registers: maximum and sum of a row need one
// exchange between two lanes, and the weights lie as the next product, V^T P^T, takes
// them.  Queries and sums stay in registers.  Keys and values go through registers into
// padded rows in LDS (8-bit ones are widened on the way, once for eight waves), keys two
// tiles ahead and values one, so that a tile costs one barrier; slots of keys are looked
// up by one wave, five tiles ahead.
//
// Two waves share a SIMD, and neither the products nor the softmax may wait for the other:
// in a tile's turn the products of the next tile's keys stand between this tile's first
// weights, the products with the values between the rest, and the next maximum is formed
// behind them.  Sums are brought to a new maximum only once it is 2^kSlack times the old
// one's weight, so most tiles multiply nothing.  The order is fixed by hand: the
// compiler's own put the parts behind each other.
//
// The line of work is all row tiles of the batch, cut into equal stretches for up to 256
// workgroups: lengths are on the device, and a tile's cost differs by its place in a
// prompt.  A tile in two stretches leaves parts, which chunk_join_kernel joins.
//
// Measured: a prompt of 8192 tokens, 32 heads over 8 of 128, 575 to 611 us (0.90 to 0.96
// PF/s; a product of two 16384 matrices reaches 1.6), 2048 tokens after 129,024 4.1 to
// 4.4 ms (1.0).  A tile of 64 keys takes 3900 cycles.  The matrix instructions of a
// SIMD's two waves are 2130 of them, their 129 vector instructions and 32 exponentials each
// 1830 (at 4.9 and 8.8 cycles): nearly the sum of both, so the two waves hardly overlap.
// The eight waves' reads of keys and values are 2050 cycles of LDS (256 KB at 128 bytes a
// cycle).  How the weights are spread over the
// products, how far reads run ahead, and the waves' priorities change nothing (within 1 %).
// A row tile's start and end take 18,000.  With one tile ahead, by direct loads
// to LDS, and a tile's products all ahead of its softmax, the long one took 4.97 ms.
template <int D, bool kFp8>
__global__ __launch_bounds__((Tile<D, kFp8>::kThreads)) void chunk_attention_kernel(
    ChunkArgs a, Parts parts, FastDiv by_block, Cut cut, FastDiv by_heads, long long* stretch_of) {
  using T = Tile<D, kFp8>;
  constexpr int kSteps = D / 16;    // products along the channels
  constexpr int kBlocks = D / 32 / T::kSplit;  // 32-channel blocks of the output
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  __shared__ Shared s_line;
  __shared__ uint32_t s_again[T::kWaves];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // The wave's rows, and its part of the channels.
  const int row_wave = wave % T::kRowWaves, part_wave = wave / T::kRowWaves;
  const int G = a.Hq / a.H;
  const int jobs = a.H * cut.head_blocks;  // of a row tile
  // Neighbouring stretches on one XCD, whose workgroups then read the same keys.
  const int slots = gridDim.x;
  const int slot = (int)(blockIdx.x & 7) * (slots >> 3) + (int)(blockIdx.x >> 3);
  char* stages = lds + T::kQueries;
  int* slots_of_keys = (int*)(stages + 2 * T::kStage);

  auto cost = [&](int b) {
    const Chunk c = chunk_of(a, b);
    const Load w{c.at, c.live, cut.tokens, a.window};
    return many_rows(a, c) ? jobs * w.before(w.tiles()) : 0ll;
  };
  Line line;
  const bool work = chunk_line<T::kWaves>(a.B, slot, slots, kLeastStretch, cost, s_line, &line);

  if (tid == 0) parts.split[slot].n = 0;
  if (tid == 0 && slot == 0) *stretch_of = line.stretch;
  if (work) {
    int b = line.b;
    Chunk ch = chunk_of(a, b);
    Load w{ch.at, ch.live, cut.tokens, a.window};
    int tiles = w.tiles();
    const long long units = w.before(tiles);
    int job = (int)floor_div(line.start - line.first, units);
    long long x0 = line.start - line.first - job * units;  // first unit in tile k
    int k = w.tile_at(x0);
    x0 -= w.before(k);
    // The next tile, of the next job, of the next request with tokens.
    auto advance = [&] {
      x0 = 0;
      if (++k < tiles) return;
      k = 0;
      if (++job < jobs) return;
      job = 0;
      do {
        if (++b >= a.B) return;
        ch = chunk_of(a, b);
      } while (!many_rows(a, ch));
      w = Load{ch.at, ch.live, cut.tokens, a.window};
      tiles = w.tiles();
    };
    for (long long left = line.end - line.start; left > 0 && b < a.B; advance()) {
      const long long x1 = min(w.units(k), x0 + left);
      left -= x1 - x0;
      const Segment seg = segment_of<T::kKeys>(w.lo(k), w.hi(k), x0, x1);
      if (x0 == 0 && x1 < w.units(k) && wave == 0 && lane_anew() == 0) {
        const int xb = job % cut.head_blocks;
        Split p;
        p.row0 = (long long)(ch.row0 + k * cut.tokens) * a.Hq +
                 (long long)(job / cut.head_blocks) * G + xb * cut.heads;
        long long stretch = line.stretch;
        asm volatile("" : "+s"(stretch));
        p.before = stretch - x1;
        p.n = (int)floor_div(p.before + w.units(k) - 1, stretch) + 1;
        p.lo = w.lo(k);
        p.hi = w.hi(k);
        p.rows = min(cut.tokens, w.live - k * cut.tokens);
        p.heads = min(cut.heads, G - xb * cut.heads);
        parts.split[slot] = p;
      }
      // A stretch in the middle of a tile: how far behind the tile's first one.
      if (x0 > 0 && x1 < w.units(k) && wave == 0 && lane_anew() == 0) {
        long long stretch = line.stretch;
        asm volatile("" : "+s"(stretch));
        parts.split[slot].n = -(int)floor_div(x0 + stretch - 1, stretch);
      }
      if (seg.begin >= seg.end) continue;
      const bool all = seg.begin == seg.first && seg.end == seg.last;
      const int h = job / cut.head_blocks, xb = job - h * cut.head_blocks;
      const int len = w.at + w.live;  // keys in all
      const int32_t* table = a.table + (size_t)b * a.max_blocks;

      // The lane's row: its token and query head.
      const int lane = lane_anew();
      const int r32 = lane & 31, half = lane >> 5, r = row_wave * 32 + r32;
      // This thread's pieces of a key tile.
      const int my_key = (wave * 64 + lane) / T::kPieces, my_piece = lane % T::kPieces;
      const bool my_load = T::kTotal >= T::kThreads || wave * 64 + lane < T::kTotal;
      const int ti = fast_div(r, by_heads), hi = r - ti * cut.heads;
      const int token = k * cut.tokens + ti;
      const bool live = ti < cut.tokens && token < w.live && xb * cut.heads + hi < G;
      // Rows of q and out: from the tile's first one on.
      const size_t row0 = (size_t)(ch.row0 + k * cut.tokens) * a.Hq + (size_t)h * G + xb * cut.heads;
      auto row_of = [&](int place) {
        const int x = fast_div(place, by_heads);
        return x * a.Hq + (place - x * cut.heads);
      };
      const bf16_t* q_rows = a.q + row0 * D;
      bf16_t* out_rows = a.out + row0 * D;
      // Rows without a token see what is there, with queries of 0.
      const int limit = live ? w.at + token : 0x3fffffff;
      const int lower = live && a.window > 0 ? max(0, limit + 1 - a.window) : 0;
      auto imax = [](int x, int y) { return max(x, y); };
      auto imin = [](int x, int y) { return min(x, y); };
      const int most_limit = __builtin_amdgcn_readfirstlane(wave_reduce(live ? limit : -1, imax));
      const int least_limit = __builtin_amdgcn_readfirstlane(wave_reduce(limit, imin));
      const int least_lower = __builtin_amdgcn_readfirstlane(wave_reduce(live ? lower : 0x3fffffff, imin));
      const int most_lower = __builtin_amdgcn_readfirstlane(wave_reduce(lower, imax));

      // Staging, through registers: in tile j's turn the keys of tile j + 2 and the
      // values of tile j + 1 go into LDS and those of the tiles behind them are asked
      // for.  One wave looks up the slots of a tile's keys, a lane a key, some tiles
      // ahead (-1: not there, or behind the segment).
      constexpr int kLookup = 3;  // the wave
      const uint32_t row_bytes = (uint32_t)a.H * (T::kPieces * 16);
      const size_t mine = (size_t)h * (T::kPieces * 16) + my_piece * 16;
      const char* my_k = (const char*)a.k_cache + mine;
      const char* my_v = (const char*)a.v_cache + mine;
      const int key_end = min(len, seg.end * T::kKeys);
      auto page_of = [&](int j) {
        return table[fast_div(min(j * T::kKeys + lane, key_end - 1), by_block)];
      };
      // (Ahead of the queries' loads, as they are waited for first.)
      const int page0 = page_of(seg.begin + min(wave, 4));
      int page = page_of(seg.begin + 5);

      // Queries; a negative scale goes into their signs.
      const float ks = a.k_scale != nullptr ? a.k_scale[h] : 1.f;
      const float signed_qs = a.scale * ks * kLog2e;
      const float qs = __builtin_bit_cast(
          float, __builtin_amdgcn_readfirstlane(
                     __builtin_bit_cast(int, fmaxf(fabsf(signed_qs), 0x1p-126f))));  // logits in powers of two
      const uint32_t flip = signed_qs < 0.f ? 0x80008000u : 0u;
      Frag16 qf[T::kQueriesInLds ? 1 : kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        Frag16 x;
        x.u = u32x4{0u, 0u, 0u, 0u};
        if (live) x.u = load16(q_rows + (uint32_t)(row_of(r) * D + 16 * u + 8 * half));
#pragma unroll
        for (int i = 0; i < 4; ++i) x.u[i] ^= flip;
        if constexpr (T::kQueriesInLds) {
          if (part_wave > 0) continue;
          store16(lds + r * T::kKeyRow + (2 * u + half) * 16, x.u);
        } else {
          qf[u] = x;
        }
      }

      auto ring = [&](int j) {
        return slots_of_keys + ((j - seg.begin) & (T::kSlots - 1)) * T::kKeys;
      };
      auto put_slots = [&](int j, int page) {
        const int p = j * T::kKeys + lane;
        const bool ok = p < key_end && page >= 0 && page < a.num_blocks;
        const int row = p - fast_div(p, by_block) * a.block_size;
        if (lane < T::kKeys) ring(j)[lane] = ok ? page * a.block_size + row : -1;
      };
      auto get_slots = [&](int j, int (&slot_of)[T::kLoads]) {
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i)
          slot_of[i] = ring(j)[(my_key + i * T::kStep) & (T::kKeys - 1)];
      };
      u32x4 kreg[T::kLoads], vreg[T::kLoads];
      bool k_there[T::kLoads], v_there[T::kLoads];
      int v_slot[T::kLoads], k_slot[T::kLoads];
      auto fetch_key = [&](int i, int slot_of) {
        k_there[i] = slot_of >= 0;
        kreg[i] = load16(my_k + (size_t)(uint32_t)max(slot_of, 0) * row_bytes);
      };
      auto fetch_value = [&](int i, int slot_of) {
        v_there[i] = slot_of >= 0;
        vreg[i] = load16(my_v + (size_t)(uint32_t)max(slot_of, 0) * row_bytes);
      };
      // Zeros for keys that are not there: infinities and NaN would show through
      // weights of 0.
      auto clear = [&] {
        bool all = true;
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) all = all && k_there[i] && v_there[i];
        if (__all(all)) return;
        asm volatile("");  // a branch, and no selects, which would wait for the loads
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) {
          kreg[i] = k_there[i] ? kreg[i] : u32x4{0u, 0u, 0u, 0u};
          vreg[i] = v_there[i] ? vreg[i] : u32x4{0u, 0u, 0u, 0u};
        }
      };
      auto put = [&](char* row, const u32x4& x, auto half_precision) {
        if (!my_load) return;
        if constexpr (kFp8) {
          u32x4 first8, last8;
          widen16<decltype(half_precision)::value>(x, &first8, &last8);
          store16(row + 2 * my_piece * 16, first8);
          store16(row + (2 * my_piece + 1) * 16, last8);
        } else {
          store16(row + my_piece * 16, x);
        }
      };
      auto put_key = [&](char* st, int i, const u32x4& x) {
        put(st + (my_key + i * T::kStep) * T::kKeyRow, x, std::false_type{});
      };
      auto put_value = [&](char* st, int i, const u32x4& x) {
        put(st + T::kValuesAt + (my_key + i * T::kStep) * T::kValueRow, x, std::true_type{});
      };

      f32x16 o[kBlocks];
#pragma unroll
      for (int c = 0; c < kBlocks; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[c][i] = 0.f;
      float m = -__builtin_huge_valf(), l = 0.f;  // m: of the products, not scaled

      // Products with a tile's keys.  Their LDS reads run kAhead products ahead: left
      // to itself, the compiler waits for each read right before its product.
      constexpr int kAhead = 4, kProducts = kSteps * T::kParts;
      f32x16 s[2][T::kParts];  // of even and odd tiles of the segment
      Frag16 kf[kProducts], xf[kProducts];
      auto read_keys = [&](const char* st, int n) {
        const int t = n % T::kParts, u = n / T::kParts;
        kf[n].u = *reinterpret_cast<const u32x4*>(st + (32 * t + r32) * T::kKeyRow +
                                                  (2 * u + half) * 16);
        if constexpr (T::kQueriesInLds)
          xf[n].u = *reinterpret_cast<const u32x4*>(lds + r * T::kKeyRow + (2 * u + half) * 16);
        else
          xf[n] = qf[u];
      };
      auto product = [&](f32x16 (&to)[T::kParts], int n) {
        const int t = n % T::kParts;  // neighbours do not wait for each other
        if (n < T::kParts) {
#pragma unroll
          for (int i = 0; i < 16; ++i) to[t][i] = 0.f;
        }
        to[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[n].h, xf[n].h, to[t], 0, 0, 0);
      };
      auto all_products = [&](const char* st, f32x16 (&to)[T::kParts]) {
#pragma unroll
        for (int n = 0; n < kAhead; ++n) read_keys(st, n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
          if (n + kAhead < kProducts) read_keys(st, n + kAhead);
          product(to, n);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      const bool any_row = most_limit >= 0;
      auto read_by_wave = [&](int j) {
        const int base = j * T::kKeys;
        return any_row && base <= most_limit && base + T::kKeys > least_lower;
      };

      // (The reads of the last segment's slots and stages are behind a barrier.)
      if (wave < 5) put_slots(seg.begin + wave, page0);
      __syncthreads();
      int slot_here = ring(seg.begin)[lane & (T::kKeys - 1)];
      {
        int at[3][T::kLoads];  // slots of the first three tiles' keys
        u32x4 first[3][T::kLoads];
#pragma unroll
        for (int x = 0; x < 3; ++x) get_slots(seg.begin + x, at[x]);
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) {
          first[0][i] = load16(my_k + (size_t)(uint32_t)max(at[0][i], 0) * row_bytes);
          first[1][i] = load16(my_v + (size_t)(uint32_t)max(at[0][i], 0) * row_bytes);
          first[2][i] = load16(my_k + (size_t)(uint32_t)max(at[1][i], 0) * row_bytes);
          fetch_key(i, at[2][i]);
          fetch_value(i, at[1][i]);
        }
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) {
          const u32x4 none = {0u, 0u, 0u, 0u};
          put_key(stages, i, at[0][i] >= 0 ? first[0][i] : none);
          put_value(stages, i, at[0][i] >= 0 ? first[1][i] : none);
          put_key(stages + T::kStage, i, at[1][i] >= 0 ? first[2][i] : none);
        }
      }
      get_slots(seg.begin + 2, v_slot);
      get_slots(seg.begin + 3, k_slot);
      __syncthreads();
      if (read_by_wave(seg.begin)) all_products(stages, s[0]);
      __syncthreads();  // the first turn puts other keys there

      // Whether a row's products of a tile reach so far above m that its sums have to be
      // brought to them.
      constexpr int kValues = 16 * T::kParts;  // products of a lane
      auto above_slack = [&](float top) -> bool {
        return __any((top - m) * qs > T::kSlack || (m == -__builtin_huge_valf() && top > m));
      };
      bool check = true;  // the tile's maximum is not known, or above

      // Tile j, in stage kAt, along with the products of the next one's keys (of what
      // lies there, behind the last tile; they are not used).
      auto turn = [&](int j, auto at) {
        constexpr int kAt = decltype(at)::value;
        const int base = j * T::kKeys;
        char* st = stages + kAt * T::kStage;
        char* st_next = stages + (1 - kAt) * T::kStage;
        const uint64_t present = __ballot(lane < T::kKeys && slot_here >= 0);
        slot_here = ring(j + 1)[lane & (T::kKeys - 1)];
        if (wave == kLookup) {
          put_slots(j + 5, page);
          page = page_of(j + 6);
        }
        clear();
        auto next_slots = [&] {
#pragma unroll
          for (int i = 0; i < T::kLoads; ++i) v_slot[i] = k_slot[i];
          get_slots(j + 4, k_slot);
        };
        if (read_by_wave(j)) {
          f32x16 (&sj)[T::kParts] = s[kAt];
          f32x16 (&sn)[T::kParts] = s[1 - kAt];
          constexpr uint64_t kAll = ~0ull >> (64 - T::kKeys);
          const bool some_hidden =
              present != kAll || base + T::kKeys - 1 > least_limit || base < most_lower;
          if (check || some_hidden) {
            if (some_hidden) {
              // Bits of the keys that the row sees; the lane's begin at 4 half.
              uint64_t seen = present;
              const int above = limit - base, below = lower - base;
              seen &= above >= 63 ? ~0ull : above < 0 ? 0ull : (2ull << above) - 1;
              seen &= below <= 0 ? ~0ull : below > 63 ? 0ull : ~0ull << below;
              seen >>= 4 * half;
#pragma unroll
              for (int t = 0; t < T::kParts; ++t) {
                const uint32_t word = (uint32_t)(seen >> (32 * t));
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (!((word >> (8 * (i / 4) + i % 4)) & 1)) sj[t][i] = -__builtin_huge_valf();
              }
            }
            float top = sj[0][0];
#pragma unroll
            for (int i = 1; i < kValues; ++i) top = fmaxf(top, sj[i / 16][i % 16]);
            top = max_of_halves(top);
            if (above_slack(top)) {
              const float mn = fmaxf(m, top);
              const float keep =
                  m == -__builtin_huge_valf() ? 0.f : __builtin_amdgcn_exp2f((m - mn) * qs);
              l *= keep;
#pragma unroll
              for (int c = 0; c < kBlocks; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[c][i] *= keep;
              m = mn;
            }
          }
          const float shift = m == -__builtin_huge_valf() ? 0.f : m * qs - T::kLift;

          // The weights go between the products with the next tile's keys and the
          // first half of those with the values; the next tile's maximum goes between
          // the second half, so that only the tiles that raise it, or hide keys from
          // some row, need more.
          constexpr int kGroups = 2 * T::kParts, kSums = kGroups * kBlocks;  // of 16 keys
          constexpr int kFirst = kValues * 5 / 8;  // weights among the products with keys
          static_assert(2 * T::kLoads <= kProducts / 2 && kFirst >= 8 * (kGroups / 2), "order");
          // The weights are rounded once.  A second part, as the few-rows kernel has it,
          // would be half as many products again with the values, where the products
          // bound this: against 64 bits the results are off by 0.0021 to 0.0023 of their
          // norm, 0.0016 of which is their own rounding to bf16.  The sum l is that of
          // the weights as they were.
          union Weights {
            bf16_t e[8];
            f16_t f[8];
            bf16x8 w;
            f16x8 v;
          } pw[kGroups];
          union Values {
            s16x4 q[2];
            bf16x8 w;
            f16x8 v;
          } vf[kSums];
          const int r16 = lane & 15, g = (lane >> 4) & 1;
          auto weigh = [&](int i) {
            const float e = __builtin_amdgcn_exp2f(fmaf(sj[i / 16][i % 16], qs, -shift));
            l += e;
            if constexpr (kFp8) pw[i / 8].f[i % 8] = (f16_t)e;
            else pw[i / 8].e[i % 8] = (bf16_t)e;
          };
          auto weights = [&](int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) weigh(i);
          };
          auto read_values = [&](int n) {
            const int y = n / kBlocks, c = n % kBlocks;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int key = 16 * y + 8 * z + 4 * half + r16 / 4;
              char* from = st + T::kValuesAt + key * T::kValueRow + 64 * (kBlocks * part_wave + c) +
                           32 * g + 8 * (r16 & 3);
              vf[n].q[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4*)(uintptr_t)(lds_void*)from);
            }
          };
#pragma unroll
          for (int n = 0; n < kAhead; ++n) read_keys(st_next, n);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = 0; n < kProducts; ++n) {
            if (n + kAhead < kProducts) read_keys(st_next, n + kAhead);
            else read_values(n + kAhead - kProducts);
            product(sn, n);
            constexpr int kFetch = kProducts / 2;
            if (n < T::kLoads) put_key(st, n, kreg[n]);
            else if (n < 2 * T::kLoads) put_value(st_next, n - T::kLoads, vreg[n - T::kLoads]);
            if (n >= kFetch && n < kFetch + T::kLoads) fetch_key(n - kFetch, k_slot[n - kFetch]);
            else if (n >= kFetch + T::kLoads && n < kFetch + 2 * T::kLoads)
              fetch_value(n - kFetch - T::kLoads, v_slot[n - kFetch - T::kLoads]);
            weights(n * kFirst / kProducts, (n + 1) * kFirst / kProducts);
            __builtin_amdgcn_sched_barrier(0);
          }
          next_slots();
          float top = -__builtin_huge_valf();
#pragma unroll
          for (int n = 0; n < kSums; ++n) {
            const int y = n / kBlocks, c = n % kBlocks;
            constexpr int kHalf = kSums / 2, kRest = kValues - kFirst;
            if (n + kAhead < kSums) read_values(n + kAhead);
            if constexpr (kFp8)
              o[c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[n].v, pw[y].v, o[c], 0, 0, 0);
            else
              o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[n].w, pw[y].w, o[c], 0, 0, 0);
            if (n < kHalf) {
              weights(kFirst + n * kRest / kHalf, kFirst + (n + 1) * kRest / kHalf);
            } else {
#pragma unroll
              for (int i = (n - kHalf) * kValues / kHalf; i < (n - kHalf + 1) * kValues / kHalf; ++i)
                top = fmaxf(top, sn[i / 16][i % 16]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          check = above_slack(max_of_halves(top));
        } else {
          if (read_by_wave(j + 1)) all_products(st_next, s[1 - kAt]);
          check = true;
#pragma unroll
          for (int i = 0; i < T::kLoads; ++i) {
            put_key(st, i, kreg[i]);
            put_value(st_next, i, vreg[i]);
            fetch_key(i, k_slot[i]);
            fetch_value(i, v_slot[i]);
          }
          next_slots();
        }
        __syncthreads();
      };
#pragma unroll 1
      for (int j = seg.begin; j < seg.end; j += 2) {
        turn(j, std::integral_constant<int, 0>{});
        if (j + 1 < seg.end) turn(j + 1, std::integral_constant<int, 1>{});
      }

      // The halves of a row hold its sum in parts.  (Places are formed anew: none are
      // held through the tiles for this.)
      const int lane2 = lane_anew();
      const int r32e = lane2 & 31, halfe = lane2 >> 5, re = row_wave * 32 + r32e;
      l = sum_of_halves(l);
      float largest = 0.f;  // NaN counts as the largest
#pragma unroll
      for (int c = 0; c < kBlocks; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          largest = __builtin_elementwise_maximum(largest, fabsf(o[c][i]));
      const bool odd = live && l > 0.f && l < __builtin_huge_valf() &&
                       !(largest < __builtin_huge_valf());
      const uint64_t odd_lanes = __ballot(odd);
      uint32_t again = (uint32_t)odd_lanes | (uint32_t)(odd_lanes >> 32);
      if constexpr (T::kSplit > 1) {
        // Of all channels.
        if (lane2 == 0) s_again[wave] = again;
        __syncthreads();
        for (int x = 0; x < T::kSplit; ++x) again |= s_again[x * T::kRowWaves + row_wave];
        again = (uint32_t)__builtin_amdgcn_readfirstlane((int)again);
      }
      if (__any(l == 0.f)) {
        // No weight: nothing, also where a value is infinite or NaN.
#pragma unroll
        for (int c = 0; c < kBlocks; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[c][i] = l == 0.f ? 0.f : o[c][i];
      }
      const float vs = a.v_scale != nullptr ? a.v_scale[h] : 1.f;
      const float f = l == 0.f ? 0.f : vs / l;
      auto sink_of = [&](int place) {
        const size_t row = (size_t)row_of(place);
        Sink<D> to;
        to.out = all ? out_rows + row * D : nullptr;
        to.lse = a.lse != nullptr ? a.lse + row0 + row : nullptr;
        const size_t part = ((size_t)slot * 2 + (seg.begin == seg.first ? 1 : 0)) * T::kRows + place;
        to.o = parts.o + part * D;
        to.ml = parts.ml + part * 2;
        return to;
      };
      const bool plain = live && !((again >> r32e) & 1);
      if (live && halfe == 0 && part_wave == 0)
        sink_of(re).put_sum(l == 0.f ? -__builtin_huge_valf() : m * qs - T::kLift, l);
      if (all) {
        // Rows lie across the lanes: through LDS (all waves are done with the stages),
        // so that a store has whole rows.
        constexpr int kOutRow = 2 * D + 16, kPieces = D / 8;
        static_assert(T::kRows * kOutRow <= 2 * T::kStage, "rows fit the stages");
        char* box = stages + row_wave * 32 * kOutRow;
#pragma unroll
        for (int c = 0; c < kBlocks; ++c)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            uint2 x;
            x.x = (uint32_t)f32_to_bf16_bits(o[c][i] * f) |
                  ((uint32_t)f32_to_bf16_bits(o[c][i + 1] * f) << 16);
            x.y = (uint32_t)f32_to_bf16_bits(o[c][i + 2] * f) |
                  ((uint32_t)f32_to_bf16_bits(o[c][i + 3] * f) << 16);
            *reinterpret_cast<uint2*>(box + r32e * kOutRow + (32 * (kBlocks * part_wave + c) + 2 * i + 4 * halfe) * 2) =
                x;
          }
        const uint32_t rows = (uint32_t)__ballot(plain);
        if constexpr (T::kSplit > 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < 32 * kPieces / 64 / T::kSplit; ++i) {
          int x = (i * T::kSplit + part_wave) * 64 + lane2;
          loaded(x);  // (as r)
          const int row = x / kPieces, piece = x % kPieces;
          const u32x4 y = *reinterpret_cast<const u32x4*>(box + row * kOutRow + piece * 16);
          if ((rows >> row) & 1)
            store16(out_rows + (uint32_t)(row_of(row_wave * 32 + row) * D + piece * 8), y);
        }
      } else if (plain) {
        const Sink<D> to = sink_of(re);
#pragma unroll
        for (int c = 0; c < kBlocks; ++c)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4*>(to.o + 32 * (kBlocks * part_wave + c) + 2 * i + 4 * halfe) =
                f32x4{o[c][i] * f, o[c][i + 1] * f, o[c][i + 2] * f, o[c][i + 3] * f};
      }
      if (__builtin_expect(again != 0, 0)) {
        const int row2 = lane_anew() & 31, place = row_wave * 32 + row2;
        const bool mine = (again >> row2) & 1;
        const int at = w.at + k * cut.tokens + fast_div(place, by_heads);
        const int from = a.window > 0 ? max(0, at + 1 - a.window) : 0;
        const int first = wave_reduce(mine ? from : 0x3fffffff, [](int x, int y) { return min(x, y); });
        const int last = wave_reduce(mine ? at : -1, [](int x, int y) { return max(x, y); });
        attend_again<D, kFp8>(a, by_block, b, h, mine ? q_rows + (size_t)row_of(place) * D : nullptr,
                              flip != 0u ? -qs : qs, m * qs - T::kLift, mine ? at : -1, from,
                              max(first, seg.begin * T::kKeys), min(last + 1, seg.end * T::kKeys),
                              kBlocks * part_wave, kBlocks * (part_wave + 1), f,
                              [&](int channel, float y) {
                                if (mine) sink_of(place).put1(channel, y);
                              });
      }
    }
  }

  if (a.few == 0) clear_rows(a, wave * 64 + lane_anew());
}

// Joins what the stretches left to be joined: workgroups (x, y) with x below `many`
// stretch x of this kernel, the others those of the few-rows kernel.
template <int D, bool kFp8>
__global__ __launch_bounds__(512) void chunk_join_kernel(ChunkArgs a, Parts parts, int many,
                                                         int cut_heads, FastDiv by_heads,
                                                         const long long* stretch_of,
                                                         Parts few_parts, int few_tracks,
                                                         FastDiv by_group) {
  using T = Tile<D, kFp8>;
  // The workgroups of a tile's first stretch and of those in its middle, which leave no
  // tile of their own, have shares, in turn: a CU alone reads few bytes at once, and
  // first stretches alone may all lie on one XCD.  (40 tokens after 30,000, 33 parts a
  // row: by the first stretches' workgroups 111 us, by all 42; 32 after 8000 33 and 17.)
  if ((int)blockIdx.x >= many) {
    int slot = blockIdx.x - many;
    const int behind = max(-__builtin_amdgcn_readfirstlane(few_parts.split[slot].n), 0);
    slot -= behind;
    const Split p = split_of(few_parts.split + slot);
    if (p.n == 0) return;
    const int share = blockIdx.y * (p.n - 1) + behind, shares = (p.n - 1) * gridDim.y;
    const int G = a.Hq / a.H, all_rows = 16 * few_tracks;
    join_rows<D, 8, 8, 1>(
        a, few_parts, all_rows, p.n, share, shares,
        [&](int r, int i) -> long long {
          return (((long long)slot + i) * 2 + (i == 0)) * all_rows + r;
        },
        [&](int r) -> long long {
          const int place = r % 16, token = fast_div(place, by_group);
          return place < p.rows
                     ? p.row0 + (long long)token * a.Hq + (r / 16) * G + (place - token * G)
                     : -1;
        });
    return;
  }
  int slot = blockIdx.x;
  const int behind = max(-__builtin_amdgcn_readfirstlane(parts.split[slot].n), 0);
  slot -= behind;
  const Split p = split_of(parts.split + slot);
  if (p.n == 0) return;
  const int share = blockIdx.y * (p.n - 1) + behind, shares = (p.n - 1) * gridDim.y;
  const long long stretch = *stretch_of, size = p.hi - p.lo + kFixed;
  auto segment = [&](int i) {
    return segment_of<T::kKeys>(p.lo, p.hi, max(stretch * i - p.before, 0ll),
                                min(stretch * (i + 1) - p.before, size));
  };
  // (One stretch may hold all of the keys: it wrote the rows itself.)
  bool whole = false;
  for (int i = 0; i < p.n; ++i) {
    const Segment s = segment(i);
    whole = whole || (s.begin == s.first && s.end == s.last);
  }
  if (whole) return;
  join_rows<D, 8, 4, 2>(
      a, parts, T::kRows, p.n, share, shares,
      [&](int r, int i) -> long long {
        const Segment s = segment(i);
        return s.begin < s.end ? ((long long)(slot + i) * 2 + (s.begin == s.first)) * T::kRows + r
                               : -1;
      },
      [&](int r) -> long long {
        const int ti = fast_div(r, by_heads), hi = r - ti * cut_heads;
        return ti < p.rows && hi < p.heads ? p.row0 + (long long)ti * a.Hq + hi : -1;
      });
}

namespace {

// The workgroups of a call, 0 of a kernel that such calls never launch.  By the sizes
// alone, not by the launch rule: a call of fewer tokens or requests, or over a shorter
// table, has no more, so that its scratch fits the other's.
struct Groups {
  int many, few;
};
int rows_of(int D) { return 32 * (D == 256 ? 4 : 8); }
Groups groups_of(int T, int B, int Hq, int H, int D, long long most) {
  const int G = Hq / H;
  const Cut cut = cut_of(G, rows_of(D));
  const double tiles = std::min(T, T / cut.tokens + B);  // of rows
  Groups g{0, 0};
  if ((long long)T * G > kFewRows)
    g.many = groups_for(tiles * H * cut.head_blocks * (most + kFixed), kLeastStretch, kCus);
  if (G <= kFewRows) g.few = chunk_few_groups(T, B, H, D, most);
  return g;
}

size_t part_rows(int groups, int D) { return (size_t)groups * 2 * rows_of(D); }

size_t many_floats(int groups, int D) {
  return groups == 0 ? 0 : 64 + split_floats(groups) + part_rows(groups, D) * (2 + D);
}

// Requests of few rows (single tokens, drafts) are read by the few-rows kernel, whose
// waves go through keys of their own, where such requests are most: where the rows of
// the batch, whose lengths the host does not know, are on average as few.  A token of
// more query heads to a key head than that is no request of few rows.  (64 requests of a
// token after 500 to 2000, 32 heads over 1: 36 us, and 42 with a launch that finds nothing
// and its places in the join.)
template <int D, bool kFp8>
hipError_t launch_cfg(ChunkArgs a, hipStream_t stream) {
  using T = Tile<D, kFp8>;
  static std::atomic<unsigned long long> done{0};
  hipError_t e = once_per_device(done, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(chunk_attention_kernel<D, kFp8>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
  });
  if (e != hipSuccess) return e;
  const int G = a.Hq / a.H;
  const long long rows = (long long)a.T * G;
  a.few = G <= kFewRows && (rows <= (long long)kFewRows * a.B || a.B >= kFewRequests) ? kFewRows : 0;
  const Groups groups = groups_of(a.T, a.B, a.Hq, a.H, D, (long long)a.max_blocks * a.block_size);
  const Parts few_parts = chunk_few_parts(a.part + many_floats(groups.many, D), groups.few, a.H);
  // The stretch, then what was split, then the parts.
  long long* stretch = (long long*)a.part;
  Parts parts;
  parts.split = (Split*)(a.part + 64);
  parts.ml = a.part + 64 + split_floats(groups.many);
  parts.o = parts.ml + part_rows(groups.many, D) * 2;
  const Cut cut = cut_of(G, T::kRows);
  const FastDiv by_heads = make_fast_div(cut.heads);
  int many = 0, few = 0;
  if (a.few > 0) {
    few = groups.few;
    e = launch_chunk_few(a, few_parts, few, stream);
    if (e != hipSuccess) return e;
  }
  if (a.few == 0 || rows > kFewRows) {
    many = groups.many;
    chunk_attention_kernel<D, kFp8><<<many, T::kThreads, T::kLds, stream>>>(
        a, parts, make_fast_div(a.block_size), cut, by_heads, stretch);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  chunk_join_kernel<D, kFp8><<<dim3(many + few, 8), 512, 0, stream>>>(
      a, parts, many, cut.heads, by_heads, stretch, few_parts, chunk_few_tracks(a.H), make_fast_div(G));
  return hipGetLastError();
}

}  // namespace

size_t chunk_scratch_floats(int T, int B, int Hq, int H, int D, long long most) {
  if (T == 0 || B == 0) return 0;
  const Groups g = groups_of(T, B, Hq, H, D, most);
  return many_floats(g.many, D) + (g.few == 0 ? 0 : chunk_few_floats(g.few, H, D));
}

hipError_t launch_chunk_attention(const ChunkArgs& a, hipStream_t stream) {
  const bool fp8 = a.dtype == kCacheFp8;
  switch (a.D) {
    case 64: return fp8 ? launch_cfg<64, true>(a, stream) : launch_cfg<64, false>(a, stream);
    case 128: return fp8 ? launch_cfg<128, true>(a, stream) : launch_cfg<128, false>(a, stream);
    case 256: return fp8 ? launch_cfg<256, true>(a, stream) : launch_cfg<256, false>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mova

// Attention of one new token per request over the paged key-value cache
// (page "MoVA: routing the value vectors ...", section "Where the routing
// happens": 32 query heads over 8 key heads of 128; the cache holds ordinary
// key and routed value vectors).
//
//   out_i = sum_p exp(s_ip - m_i) v_p / sum_p exp(s_ip - m_i),  s_ip = scale q_i . k_p
//
// in one pass over the keys with the running maximum m and sum of a softmax.
// A key and its value are read once for the group of query heads that share
// them: 4 flops a byte at a group of 4, so the kernel is bound by reading the
// cache, and everything below serves that stream.
//
// Work: the keys of a request, per group of key heads, are cut into tiles.
// All tiles of the batch lie in one line, request after request, and each of
// the workgroups (one or two per CU) takes an equal stretch of it, so ragged
// batches and single long requests fill the chip alike and the host needs no
// lengths.  A request whose tiles lie in one stretch is finished there; else
// each stretch leaves its part (m, sum, unnormalised out; fp32) in the
// workspace and attention_join_kernel adds them.  Where no row can have more
// than a few tiles the line is one of whole rows (`whole`).  With a list, the
// tiles are those of as many of its entries as the request has blocks.
//
// A workgroup's four waves take four tracks (a key head with up to 16 of its
// query heads) at the same positions (rows of 4 x head_dim elements are
// contiguous), or stripes of the tiles where there are fewer.  Each wave is a
// pipeline of its own: a ring of tiles in LDS, filled by direct-to-LDS loads
// with kStages - 1 tiles in flight while one is used; no barrier but at the
// ends.  The block table (and the list of chosen blocks) is fetched the same
// way, kStages tiles ahead of the tile whose addresses need it.
//
// A tile's logits are MFMA products K Q^T (16 keys x 16 query heads, heads
// past the group are zero), so a lane holds four keys of one query head and
// the softmax needs two lane exchanges a tile.  Their weights are then, as
// they lie in the registers, the second operand of out^T = V^T P^T, whose
// first operand the transposing LDS reads deliver; the sums over keys may run
// in any order as long as both operands agree.  Weights go into this product
// as two bf16 parts (2^-16 relative), and the others of the softmax stay fp32.
// Against the 64-bit result rounded to bf16 that leaves 0.2 % of the elements
// one step off (64 requests of 500 to 8000 tokens; 0.05 % with fp32 weights); a
// third part cost 8-bit caches 1.4 % of their time.  8-bit elements are widened
// to bf16, which is exact.
#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "paged.h"

namespace mova {

// Numbers of the line of tiles that the join needs: prefix[b] is the first
// tile of request b, prefix[B] the tiles of a stretch.
struct Parts {
  long long* prefix;
  float* ml;  // [two a workgroup][tracks per group][rows][2]
  float* o;   // [two a workgroup][tracks per group][rows][D]
};

namespace {

constexpr int kCus = 256;
constexpr int kMaxGrid = 2 * kCus;  // workgroups of attention_kernel

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2;

// A track is a key head with up to 16 of the query heads that share it.
int tracks_of(int Hq, int H) { return H * ceil_div(Hq / H, 16); }
// Waves of a workgroup on different tracks; the others split the tiles.
int tracks_per_group(int tracks) { return tracks % 4 == 0 ? 4 : tracks % 2 == 0 ? 2 : 1; }

template <int D, bool kFp8>
struct Tile {
  static constexpr int kBytes = kFp8 ? 1 : 2;                   // of an element
  static constexpr int kKeys = (!kFp8 && D >= 128) ? 16 : 32;   // of a tile
  static constexpr int kRow = D * kBytes;                       // bytes of a key
  static constexpr int kChunks = kRow / 16;                     // 16-byte pieces of a key
  static constexpr int kRowsPerLoad = 64 / kChunks;
  static constexpr int kLoads = kKeys / kRowsPerLoad;           // wave loads per side
  static constexpr int kSide = kKeys * kRow;                    // bytes of a side (K or V)
  // Two workgroups a CU with 16 KB of keys and values a wave, or one with 32:
  // two hide each other's softmax and beginnings, where two tiles fit 16 KB (64
  // requests of 500 to 8000 tokens: 8 heads of 128 122.0 -> 121.5 us, of 64 66.5
  // -> 66.0; 8 bits, 8 heads of 64 52.8 -> 44.4, 3 heads of 128 39.4 -> 32.9).
  static constexpr int kPerCu = 4 * kSide <= 16384 ? 2 : 1;
  static constexpr int kRing = 32768 / kPerCu;
  static constexpr int kStages = kRing / (2 * kSide);
  static constexpr int kLds = kRing + 2 * kStages * 256;        // with the block numbers
  // The non-temporal hint, where a row fills a 128-byte cache line (the same
  // batch, 8 heads of 128: 138 -> 121 us, of 64: 75 -> 66); two heads' waves share
  // the line of a shorter row, and the hint would have it read twice (64 wide with
  // 8 bits: 44 us without, 53 with).
  static constexpr bool kStream = kRow >= 128;
  static_assert(kStages >= 2 && kChunks <= 32 && kRowsPerLoad >= 2, "tile shape");
  // Piece c of row r lies at piece c ^ swizzle(r), so that the 8 rows of one
  // phase of the key fragments' reads, and the rows that 16 lanes of a
  // transposing read take, fall into different banks.
  static __device__ __forceinline__ int swizzle_k(int r) {
    constexpr int kShare = kChunks >= 8 ? 1 : 8 / kChunks;
    return (r / kShare) & (kChunks - 1) & 15;
  }
  static __device__ __forceinline__ int swizzle_v(int r) {
    constexpr int kShare = kChunks >= 16 ? 1 : 16 / kChunks;
    if constexpr (!kFp8) return (2 * (r / kShare)) & (kChunks - 1) & 15;
    else if constexpr (kChunks == 4) return ((r >> 4) & 1) | ((r >> 1) & 2);
    else if constexpr (kChunks == 8) return ((r >> 1) & 1) | ((r >> 3) & 2) | (r & 4);
    else return (r & 3) | ((r >> 2) & 4) | ((r << 1) & 8);
  }
};

size_t prefix_floats(int B) { return ((size_t)(B + 1) * 2 + 63) / 64 * 64; }

Parts parts_of(const AttentionArgs& a) {
  const size_t rows = (size_t)kMaxGrid * 2 * tracks_per_group(tracks_of(a.Hq, a.H)) * std::min(a.Hq / a.H, 16);
  Parts p;
  p.prefix = (long long*)a.part;
  p.ml = a.part + prefix_floats(a.B);
  p.o = p.ml + (rows * 2 + 63) / 64 * 64;
  return p;
}

// Keys request b reads, [lo, lo + keys) or, with a list, those of its first
// entries, as many as the request has blocks: all there is where each block is
// listed once and ahead of the entries that name none.  What is listed behind
// them belongs to the row's last tile.
struct Span {
  int len, lo;
  int keys;
};
__device__ __forceinline__ Span span_of(const AttentionArgs& a, int b) {
  Span s;
  s.len = a.num_blocks > 0 ? request_len(a.seq_lens, b, a.max_blocks, a.block_size) : 0;
  s.lo = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.keys = a.sel != nullptr ? min(a.keep, ceil_div(s.len, a.block_size)) * a.block_size
                            : s.len - s.lo;
  return s;
}

// Sums of weighted values above kMostSum (or not finite) are formed once more,
// with weights relative to 2^kLift times the largest.  The second pass cannot
// overflow, as a row has at most 2^30 keys, nor can the sums of its parts with
// those of the others (at most 4 * 2 * kMaxGrid of them, each up to kMostSum).
// And a weight's second part, 0 or negative for many, is kept at 2^-22 of the
// weight or more, so that its product with an infinite value is that infinity.
// (The first part is cut rather than rounded for that, which costs it a bit.)
constexpr float kMostSum = 0x1p112f, kLift = 31.f, kLeastPart = 0x1p-22f;

// 8 e4m3 elements as bf16 (exact).
__device__ __forceinline__ Frag16 widen_fp8(uint32_t w0, uint32_t w1) {
  auto two = [](uint32_t w, auto upper) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                            (int)w, 1.f, decltype(upper)::value));
  };
  Frag16 f;
  f.u = u32x4{two(w0, std::false_type{}), two(w0, std::true_type{}), two(w1, std::false_type{}),
              two(w1, std::true_type{})};
  return f;
}

// Largest of the lanes i, i + 16, i + 32 and i + 48, in all of them: exchanges of
// rows of 16 and of halves in registers.
__device__ __forceinline__ float max_over_groups(float x) {
  uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto rows = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = fmaxf(__builtin_bit_cast(float, (uint32_t)rows[0]), __builtin_bit_cast(float, (uint32_t)rows[1]));
  u = __builtin_bit_cast(uint32_t, x);
  const auto halves = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)halves[0]),
               __builtin_bit_cast(float, (uint32_t)halves[1]));
}

// Four transposing LDS reads of 8 bytes a lane (16 lanes hand out 16 columns of
// the 128 bytes that they address) and the wait for them, in one block: as
// builtins, each read would first wait for every direct load in flight (the
// compiler cannot tell which part of the ring those fill), which would empty
// the pipeline.
template <bool kFp8>
__device__ __forceinline__ void read4_transposed(i32x2 (&v)[4], const uint32_t (&at)[4]) {
  if constexpr (kFp8)
    asm volatile(
        "ds_read_b64_tr_b8 %0, %4\n\tds_read_b64_tr_b8 %1, %5\n\t"
        "ds_read_b64_tr_b8 %2, %6\n\tds_read_b64_tr_b8 %3, %7\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
        : "memory");
  else
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %5\n\t"
        "ds_read_b64_tr_b16 %2, %6\n\tds_read_b64_tr_b16 %3, %7\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
        : "memory");
}

}  // namespace

// kTracks: tracks of a workgroup; 4 / kTracks waves share a track's tiles.
// kShared: tracks of one key head lie side by side and read the same rows.
template <int D, bool kFp8, int kTracks, bool kShared, bool kList>
__global__ __launch_bounds__(256) void attention_kernel(AttentionArgs a, Parts parts,
                                                        FastDiv by_block, int whole) {
  using T = Tile<D, kFp8>;
  constexpr int kStripes = 4 / kTracks;
  constexpr bool kStream = T::kStream && !kShared;
  constexpr int S = T::kStages;
  constexpr int kSub = T::kKeys / 16;      // 16-key parts of a tile
  constexpr int kCols = D / 16;
  constexpr int kGroupLoads = 2 * T::kLoads + (kList ? 2 : 1);
  static_assert((S - 1) * kGroupLoads < 64, "outstanding loads");
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  __shared__ LineShared s_line;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int tsub = wave / kStripes, stripe = wave % kStripes;
  const int G = a.Hq / a.H;
  const int qtiles = ceil_div(G, 16);
  const int rows_per_b = a.H * qtiles / kTracks;
  char* ring = lds + wave * T::kLds;
  int* pages = (int*)(ring + T::kRing);
  int* listed = pages + S * 64;

  // Units of the line that a request brings: its tiles, or its rows.
  auto tiles_of = [&](const Span& s) { return ceil_div(s.keys, T::kKeys * kStripes); };
  auto units_of = [&](int n) { return (long long)(whole ? 1 : n) * rows_per_b; };
  Line line;
  if (!line_begin(a.B, [&](int b) { return units_of(whole ? 0 : tiles_of(span_of(a, b))); }, s_line,
                  parts.prefix, &line))
    return;

  const uint32_t row_bytes = (uint32_t)a.H * T::kRow;
  int b = line.b;
  long long at = line.first;  // first tile of request b
  Span sp = span_of(a, b);
  int n = tiles_of(sp);
  bool again = false;  // the second pass over a row's share
  for (long long pos = line.start; pos < line.end;) {
    while (pos >= at + units_of(n)) {
      at += units_of(n);
      if (++b >= a.B) return;
      sp = span_of(a, b);
      n = tiles_of(sp);
    }
    const int row = whole ? (int)(pos - at) : (int)floor_div(pos - at, n);
    const int t0 = whole ? 0 : (int)(pos - at - (long long)row * n);
    const int t1 = whole ? n : (int)min((long long)n, t0 + (line.end - pos));
    pos += whole ? 1 : t1 - t0;
    const int track = row * kTracks + tsub;
    const int h = track / qtiles, qt = track - h * qtiles;
    int nt = t1 - t0;
    const bool all = nt == n;
    const int blocks = ceil_div(sp.len, a.block_size);
    const int32_t* table = a.table + (size_t)b * a.max_blocks;
    const int32_t* list = kList ? a.sel + ((size_t)b * a.H + h) * a.keep : nullptr;
    const int rows = min(G - qt * 16, 16);
    const bool has_row = r16 < rows;
    const size_t qrow = (size_t)b * a.Hq + h * G + qt * 16 + r16;

    // The lane's key of tile x: its index in the span, its block in the span
    // or list, and its row of that block.
    auto locate = [&](int x, int* blk, int* r) {
      const int v = ((t0 + x) * kStripes + stripe) * T::kKeys + (lane & (T::kKeys - 1));
      const int p = kList ? v : sp.lo + v;
      *blk = fast_div(p, by_block);
      *r = p - *blk * a.block_size;
    };
    if (kList && t1 == n && blocks < a.keep && n > 0) {
      // Entries behind those of the span: most often none names a block.
      int last = -1, l = lane;
      loaded(l);  // no register of the main loop for what follows from it
#pragma unroll 1
      for (int i = blocks; i < a.keep; i += 256) {
        int e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = list[min(i + 64 * k + l, a.keep - 1)];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (const uint64_t there = __ballot(e[k] >= 0 && e[k] < blocks))
            last = min(i + 64 * k + 63 - __clzll((long long)there), a.keep - 1);
      }
      if (last >= 0)
        nt = __builtin_amdgcn_readfirstlane(
            max(nt, ceil_div((last + 1) * a.block_size, T::kKeys * kStripes) - t0));
    }
    auto list_address = [&](int x) {
      int blk, r;
      locate(x, &blk, &r);
      return list + min(blk, a.keep - 1);
    };
    // Table row entry to fetch for tile x; `blk` from the list in that mode.
    auto table_address = [&](int blk) { return table + min(max(blk, 0), a.max_blocks - 1); };
    auto block_of = [&](int x, int from_list) {
      int blk, r;
      locate(x, &blk, &r);
      return kList ? from_list : blk;
    };
    // Issues tile x: addresses from its block numbers, the loads of its keys
    // and values, and the fetches for later tiles.  Returns which of its keys
    // take part (bit = key).
    auto issue = [&](int x, int page, int from_list, int next_list) -> uint32_t {
      int blk, r;
      locate(x, &blk, &r);
      bool ok;
      if constexpr (kList) {
        ok = blk < a.keep && from_list >= 0 && from_list < blocks;
        const int p = (ok ? from_list : 0) * a.block_size + r;
        ok = ok && p >= sp.lo && p < sp.len;
      } else {
        ok = blk * a.block_size + r < sp.len;
      }
      ok = ok && page >= 0 && page < a.num_blocks;
      const uint32_t mask = (uint32_t)__ballot(ok) & (uint32_t)((1ull << T::kKeys) - 1);
      const int slot = ok ? page * a.block_size + r : 0;
      char* stage = ring + (x & (S - 1)) * 2 * T::kSide;
      uint32_t row_slot[T::kLoads];  // exchanged together, before the first load
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i)
        row_slot[i] = (uint32_t)__shfl(slot, i * T::kRowsPerLoad + lane / T::kChunks);
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) {
        const int rr = i * T::kRowsPerLoad + lane / T::kChunks;
        const size_t off = (size_t)row_slot[i] * row_bytes + (size_t)h * T::kRow;
        const int c = lane % T::kChunks;
        piece_to_lds<kStream>((const char*)a.k_cache + off + (c ^ T::swizzle_k(rr)) * 16,
                                 stage + i * 1024);
        piece_to_lds<kStream>((const char*)a.v_cache + off + (c ^ T::swizzle_v(rr)) * 16,
                                 stage + T::kSide + i * 1024);
      }
      word_to_lds(table_address(block_of(x + S, next_list)), pages + (x & (S - 1)) * 64);
      if constexpr (kList) word_to_lds(list_address(x + 2 * S), listed + (x & (S - 1)) * 64);
      return mask;
    };

    // Queries: with 8-bit keys a lane's 16-byte piece serves two products.
    Frag16 qf[D / 32];
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int d = kFp8 ? 64 * (u / 2) + 16 * g4 + 8 * (u & 1) : 32 * u + 8 * g4;
      qf[u].u = u32x4{0u, 0u, 0u, 0u};
      if (has_row) qf[u].u = load16(a.q + qrow * D + d);
    }
    const float ks = a.k_scale != nullptr ? a.k_scale[h] : 1.f;
    const float vs = a.v_scale != nullptr ? a.v_scale[h] : 1.f;
    const float qs = a.scale * ks * 1.44269504088896340736f;  // logits in powers of two

    uint32_t masks[S] = {};  // of the tiles in the ring
    int ahead[S] = {};       // list entries of the tiles that come into it next
    // The last segment's LDS reads are done before the ring is filled again.
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
    asm volatile("" ::: "memory");
    if constexpr (kList) {
#pragma unroll
      for (int i = 0; i < S; ++i) ahead[i] = *list_address(i);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      word_to_lds(table_address(block_of(i, ahead[i])), pages + i * 64);
      if constexpr (kList) word_to_lds(list_address(S + i), listed + i * 64);
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));
    asm volatile("" ::: "memory");

    f32x4 o[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -__builtin_huge_valf(), l = 0.f;

    // The S turns before tile 0 only fill the ring.
    for (int x = -S; x < nt; ++x) {
      const uint32_t mask = masks[0];
#pragma unroll
      for (int i = 0; i + 1 < S; ++i) masks[i] = masks[i + 1];
      // Tile x and the fetches issued with it have landed.
      if (x >= 0) wait_groups<S - 1, kGroupLoads>(min(S - 1, nt - 1 - x));
      asm volatile("" ::: "memory");
      char* stage = ring + (x & (S - 1)) * 2 * T::kSide;
      constexpr uint32_t kAll = (uint32_t)((1ull << T::kKeys) - 1);
      if (x >= 0 && mask != 0) {
        if (mask != kAll) {
          // Values that take no part become zeros: their weight is zero, but
          // what lies there may be infinite or NaN.
          constexpr int kUnroll = T::kLoads > 4 ? 1 : T::kLoads;  // a register each
#pragma unroll kUnroll
          for (int i = 0; i < T::kLoads; ++i)
            if (!((mask >> (i * T::kRowsPerLoad + lane / T::kChunks)) & 1))
              *reinterpret_cast<u32x4*>(stage + T::kSide + i * 1024 + lane * 16) =
                  u32x4{0u, 0u, 0u, 0u};
        }
        float p[kSub][4];
        float top = -__builtin_huge_valf();
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
          f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
          const int rr = 16 * t + r16;
          const char* kr = stage + rr * T::kRow;
          if constexpr (!kFp8) {
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
              Frag16 kf;
              kf.u = *reinterpret_cast<const u32x4*>(kr + ((4 * u + g4) ^ T::swizzle_k(rr)) * 16);
              s = mfma16x16x32(kf.h, qf[u].h, s);
            }
          } else {
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
              const u32x4 w =
                  *reinterpret_cast<const u32x4*>(kr + ((4 * u + g4) ^ T::swizzle_k(rr)) * 16);
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const Frag16 kf = widen_fp8(w[2 * half], w[2 * half + 1]);
                s = mfma16x16x32(kf.h, qf[2 * u + half].h, s);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) p[t][i] = s[i] * qs;
        }
        if (mask != kAll) {
          const uint32_t of_lane = mask >> (4 * g4);
#pragma unroll
          for (int t = 0; t < kSub; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((of_lane >> (16 * t + i)) & 1)) p[t][i] = -__builtin_huge_valf();
        }
#pragma unroll
        for (int t = 0; t < kSub; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, p[t][i]);
        top = max_over_groups(top) + (again ? kLift : 0.f);
        const float mn = fmaxf(m, top);
        const float safe = mn == -__builtin_huge_valf() ? 0.f : mn;
        if (__any(mn > m)) {
          const float keep = __builtin_amdgcn_exp2f(m - safe);
          l *= keep;
#pragma unroll
          for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][i] *= keep;
        }
        m = mn;
        // The weights in two bf16 parts, w = high + low to 2^-16: with 16-key
        // tiles both parts fill one product's operand, against the same values
        // twice; with 32-key tiles they are two products.
        union PFrag {
          bf16_t e[8];
          s16x4 h[2];
          bf16x8 w;
        } high, low;
#pragma unroll
        for (int t = 0; t < kSub; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = __builtin_amdgcn_exp2f(p[t][i] - safe);
            l += e;
            const uint32_t bits = __builtin_bit_cast(uint32_t, e) & (again ? 0xffff0000u : ~0u);
            high.e[4 * t + i] = (bf16_t)__builtin_bit_cast(float, bits);
            const float rest = e - (float)high.e[4 * t + i];
            low.e[4 * t + i] = (bf16_t)(kFp8 ? rest : fmaxf(rest, e * (again ? kLeastPart : -1.f)));
          }
        if constexpr (kSub == 1) high.h[1] = low.h[0];
        const uint32_t vt = (uint32_t)(uintptr_t)(lds_void*)(stage + T::kSide);
        constexpr int kPer = kFp8 ? 1 : kSub;  // reads a 16-column part
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 4 / kPer) {
          uint32_t from[4];
          i32x2 got[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + i / kPer, t = i % kPer;
            const int rr =
                kFp8 ? 4 * g4 + (r16 / 2 & 3) + 16 * (r16 / 8) : 16 * t + 4 * g4 + r16 / 4;
            const int piece = kFp8 ? c : 2 * c + (r16 & 3) / 2;
            from[i] = vt + rr * T::kRow + (piece ^ T::swizzle_v(rr)) * 16 + 8 * (r16 & 1);
          }
          read4_transposed<kFp8>(got, from);
#pragma unroll
          for (int i = 0; i < 4 / kPer; ++i) {
            f32x4& acc = o[c0 + i];
            if constexpr (kFp8) {
              const Frag16 vf = widen_fp8((uint32_t)got[i][0], (uint32_t)got[i][1]);
              acc = mfma16x16x32(vf.h, high.w, acc);
              acc = mfma16x16x32(vf.h, low.w, acc);
            } else {
              PFrag vf;
              vf.h[0] = __builtin_bit_cast(s16x4, got[kSub * i]);
              vf.h[1] = __builtin_bit_cast(s16x4, got[kSub * i + kSub - 1]);
              acc = mfma16x16x32(vf.w, high.w, acc);
              if constexpr (kSub == 2) acc = mfma16x16x32(vf.w, low.w, acc);
            }
          }
        }
      }
      if (x + S < nt) {
        // Tile x + S takes this tile's place; the block numbers of it (and
        // the list entries of tile x + 2 S) came with tile x.
        const int page = pages[(x & (S - 1)) * 64 + lane];
        const int nxt = kList ? listed[(x & (S - 1)) * 64 + lane] : 0;
        const int cur = ahead[0];
#pragma unroll
        for (int i = 0; i + 1 < S; ++i) ahead[i] = ahead[i + 1];
        ahead[S - 1] = nxt;
        __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
        asm volatile("" ::: "memory");
        masks[S - 1] = issue(x + S, page, cur, nxt);
      }
    }

    // The four lanes of a query head hold its sum in parts.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if constexpr (!kFp8) {  // (8-bit values are at most 448)
      float most = 0.f;     // NaN counts as the largest
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) most = __builtin_elementwise_maximum(most, fabsf(o[c][i]));
      again = !again && __any(has_row && !(most < kMostSum) && l > 0.f && l < __builtin_huge_valf());
      if (again) {
        pos -= whole ? 1 : t1 - t0;
        continue;
      }
    }
    if (__any(l == 0.f)) {
      // No weight: nothing, also where a value is infinite or NaN.
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[c][i] = l == 0.f ? 0.f : o[c][i];
    }
    if constexpr (kStripes > 1) {
      // Stripes of a head meet in its first wave, through the ring.
      __syncthreads();
      float* box = (float*)(lds + wave * T::kLds);
#pragma unroll
      for (int c = 0; c < kCols; ++c) *reinterpret_cast<f32x4*>(box + (c * 64 + lane) * 4) = o[c];
      float* ml = (float*)(ring + T::kRing);
      ml[lane] = m;
      ml[64 + lane] = l;
      __syncthreads();
      if (stripe == 0) {
#pragma unroll 1
        for (int s = 1; s < kStripes; ++s) {
          const char* other = lds + (wave + s) * T::kLds;
          const float* oml = (const float*)(other + T::kRing);
          const float m2 = oml[lane], l2 = oml[64 + lane];
          const float mn = fmaxf(m, m2);
          const float safe = mn == -__builtin_huge_valf() ? 0.f : mn;
          const float e1 = __builtin_amdgcn_exp2f(m - safe), e2 = __builtin_amdgcn_exp2f(m2 - safe);
          l = l * e1 + l2 * e2;
          m = mn;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const f32x4 o2 = *reinterpret_cast<const f32x4*>((const float*)other + (c * 64 + lane) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][i] = o[c][i] * e1 + o2[i] * e2;
          }
        }
      }
      __syncthreads();
      if (stripe != 0) continue;
    }
    if (!has_row) continue;
    if (all) {
      const float f = l == 0.f ? 0.f : vs / l;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        uint2 w;
        w.x = (uint32_t)f32_to_bf16_bits(o[c][0] * f) | ((uint32_t)f32_to_bf16_bits(o[c][1] * f) << 16);
        w.y = (uint32_t)f32_to_bf16_bits(o[c][2] * f) | ((uint32_t)f32_to_bf16_bits(o[c][3] * f) << 16);
        *reinterpret_cast<uint2*>(a.out + qrow * D + 16 * c + 4 * g4) = w;
      }
      if (a.lse != nullptr && g4 == 0)
        a.lse[qrow] = l == 0.f ? -__builtin_huge_valf()
                               : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
    } else {
      const int cap = min(G, 16);
      const size_t part = ((size_t)(blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * kTracks + tsub) * cap + r16;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        *reinterpret_cast<f32x4*>(parts.o + part * D + 16 * c + 4 * g4) = o[c];
      if (g4 == 0) {
        parts.ml[2 * part] = m;
        parts.ml[2 * part + 1] = l;
      }
    }
  }
}

// Adds the parts of a request's query heads that were split over stretches, and
// writes the rows of requests without keys.  Workgroup (x, request) has
// kAtOnce query heads (1 or 4).  A head of few parts is one wave's work, with
// one memory round trip and no barrier; one of many (a long request in few) is
// several workgroups', a slice of its channels each.
template <int D, int kAtOnce>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, Parts parts, int tracks,
                                                             int tile_keys) {
  constexpr int kPer = D / 64;      // channels of a lane
  constexpr int kFew = 32, kBatch = 8;
  // (Four heads a workgroup: rarely many parts, and registers are waves at once.)
  constexpr int kManyBatch = kAtOnce == 1 ? 8 : 1;
  constexpr int kSlice = 32;        // channels of a workgroup of a head of many parts
  constexpr int kSlots = kMaxGrid / 256;
  typedef __attribute__((__vector_size__(kPer * sizeof(float)))) float vec;
  typedef __attribute__((__vector_size__(kPer * sizeof(__bf16)))) __bf16 half_vec;
  typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
  __shared__ float s_e[kMaxGrid], s_m[4], s_l[4];
  __shared__ f32x4 s_o[4][8];
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = ceil_div(span_of(a, b).keys, tile_keys);
  const long long stretch = parts.prefix[a.B], before = parts.prefix[b];
  const int G = a.Hq / a.H;
  const int qtiles = ceil_div(G, 16), cap = min(G, 16);

  auto scale_of = [&](int hq, float sum) {
    return (a.v_scale != nullptr ? a.v_scale[hq / G] : 1.f) / sum;
  };
  auto write_lse = [&](int hq, float sum, float safe) {
    if (a.lse != nullptr)
      a.lse[(size_t)b * a.Hq + hq] =
          sum == 0.f ? -__builtin_huge_valf()
                     : (safe + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
  };
  auto finish = [&](int hq, vec o, float sum, float safe) {
    const float f = scale_of(hq, sum);
    half_vec y;
#pragma unroll
    for (int j = 0; j < kPer; ++j) y[j] = (__bf16)(sum == 0.f ? 0.f : o[j] * f);
    *reinterpret_cast<half_vec*>(a.out + ((size_t)b * a.Hq + hq) * D + kPer * lane) = y;
    if (lane == 0) write_lse(hq, sum, safe);
  };
  // First part of the head, and how many there are.
  auto parts_at = [&](int hq, int* w0) {
    const int h = hq / G, gi = hq - h * G;
    const long long first = before + (long long)((h * qtiles + gi / 16) / tracks) * n;
    *w0 = (int)floor_div(first, stretch);
    return n == 0 ? 0 : min((int)floor_div(first + n - 1, stretch), kMaxGrid - 1) - *w0 + 1;
  };
  auto part_of = [&](int hq, int w0, int i) {
    const int h = hq / G, gi = hq - h * G;
    return ((size_t)((w0 + i) * 2 + (i == 0 ? 1 : 0)) * tracks + (h * qtiles + gi / 16) % tracks) * cap +
           gi % 16;
  };
  auto larger = [](float p, float q) { return fmaxf(p, q); };

  if (blockIdx.z == 0) {
    const int hq = blockIdx.x * kAtOnce + wave;
    int w0;
    const int np = wave < kAtOnce && hq < a.Hq ? parts_at(hq, &w0) : 1;
    if (np == 0) finish(hq, vec{}, 0.f, 0.f);
    if (np > 1 && np <= kFew) {
      // Everything is asked for before the first wait.
      float m = -__builtin_huge_valf(), l = 0.f;
      if (lane < np) {
        const float2 v = *reinterpret_cast<const float2*>(parts.ml + 2 * part_of(hq, w0, lane));
        m = v.x;
        l = v.y;
      }
      vec x[kBatch], o = {};
      auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k < np)
            x[k] = *reinterpret_cast<const vec*>(parts.o + part_of(hq, w0, i0 + k) * D + kPer * lane);
      };
      load(0);
      const float M = wave_reduce(m, larger);
      const float safe = M == -__builtin_huge_valf() ? 0.f : M;
      const float e = __builtin_amdgcn_exp2f(m - safe);
      const float sum = wave_sum(l * e);
      for (int i0 = 0; i0 < np; i0 += kBatch) {
        if (i0 != 0) load(i0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k < np) {
            const float f = __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, e), i0 + k));
#pragma unroll
            for (int j = 0; j < kPer; ++j) o[j] += x[k][j] * f;
          }
      }
      finish(hq, o, sum, safe);
    }
  }

  for (int t = 0; t < kAtOnce; ++t) {
    const int hq = blockIdx.x * kAtOnce + t;
    int w0 = 0;
    const int np = hq < a.Hq ? parts_at(hq, &w0) : 0;  // at most kMaxGrid
    if (np <= kFew) continue;
    float m[kSlots], l[kSlots], M = -__builtin_huge_valf();
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      m[k] = -__builtin_huge_valf();
      l[k] = 0.f;
      if (tid + 256 * k < np) {
        const float2 v =
            *reinterpret_cast<const float2*>(parts.ml + 2 * part_of(hq, w0, tid + 256 * k));
        m[k] = v.x;
        l[k] = v.y;
      }
      M = fmaxf(M, m[k]);
    }
    // A wave's load is a slice of eight parts.
    const int sub = 8 * wave + lane / 8;
    f32x4 x[kManyBatch];
    auto load = [&](int c, int i0) {
#pragma unroll
      for (int k = 0; k < kManyBatch; ++k)
        if (i0 + 32 * k + sub < np)
          x[k] = *reinterpret_cast<const f32x4*>(
              parts.o + part_of(hq, w0, i0 + 32 * k + sub) * D + c + 4 * (lane & 7));
    };
    load(kSlice * blockIdx.z, 0);
    M = wave_reduce(M, larger);
    if (lane == 0) s_m[wave] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    const float safe = M == -__builtin_huge_valf() ? 0.f : M;
    // Sums in a fixed order: a thread's, over the lanes, then the waves.
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const float e = __builtin_amdgcn_exp2f(m[k] - safe);
      s_e[tid + 256 * k] = e;
      sum += l[k] * e;
    }
    sum = wave_sum(sum);
    if (lane == 0) s_l[wave] = sum;
    __syncthreads();
    sum = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
    for (int c = kSlice * blockIdx.z; c < D; c += kSlice * gridDim.z) {
      f32x4 o = {};
      for (int i0 = 0; i0 < np; i0 += 32 * kManyBatch) {
        if (i0 != 0 || c != (int)(kSlice * blockIdx.z)) load(c, i0);
#pragma unroll
        for (int k = 0; k < kManyBatch; ++k)
          if (i0 + 32 * k + sub < np) {
            const float f = s_e[i0 + 32 * k + sub];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += x[k][j] * f;
          }
      }
#pragma unroll
      for (int step = 8; step < 64; step *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], step);
      if (lane < 8) s_o[wave][lane] = o;
      __syncthreads();
      if (tid < 8) {
        o = (s_o[0][tid] + s_o[1][tid]) + (s_o[2][tid] + s_o[3][tid]);
        const float f = scale_of(hq, sum);
        bf16x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = (__bf16)(sum == 0.f ? 0.f : o[j] * f);
        *reinterpret_cast<bf16x4*>(a.out + ((size_t)b * a.Hq + hq) * D + c + 4 * tid) = y;
      }
      __syncthreads();
    }
    if (tid == 0 && blockIdx.z == 0) write_lse(hq, sum, safe);
  }
}

size_t attention_scratch_floats(int B, int Hq, int H, int D) {
  if (B == 0) return 0;
  const size_t rows = (size_t)kMaxGrid * 2 * tracks_per_group(tracks_of(Hq, H)) * std::min(Hq / H, 16);
  return prefix_floats(B) + (rows * 2 + 63) / 64 * 64 + rows * D;
}

namespace {

// Keys of a row at most.
long long most_keys(const AttentionArgs& a) {
  if (a.sel != nullptr) return (long long)std::min(a.keep, a.max_blocks) * a.block_size;
  const long long keys = (long long)a.max_blocks * a.block_size;
  return a.window > 0 ? std::min<long long>(keys, a.window) : keys;
}

template <int D, bool kFp8, int kTracks, bool kShared, bool kList>
hipError_t launch_cfg(const AttentionArgs& a, bool whole, hipStream_t stream) {
  using T = Tile<D, kFp8>;
  static std::atomic<unsigned long long> done{0};
  hipError_t e = once_per_device(done, [&] {
    return hipFuncSetAttribute(
        reinterpret_cast<const void*>(attention_kernel<D, kFp8, kTracks, kShared, kList>),
        hipFuncAttributeMaxDynamicSharedMemorySize, 4 * T::kLds);
  });
  if (e != hipSuccess) return e;
  const Parts parts = parts_of(a);
  const int tile_keys = T::kKeys * (4 / kTracks);
  attention_kernel<D, kFp8, kTracks, kShared, kList>
      <<<T::kPerCu * kCus, 256, 4 * T::kLds, stream>>>(a, parts, make_fast_div(a.block_size), whole);
  e = hipGetLastError();
  if (e != hipSuccess || whole) return e;
  // Few heads in the batch may have many parts each: a workgroup a head, and
  // as many as keep the launch short a slice.
  const int heads = a.B * a.Hq;
  if (heads >= 1024) {
    attention_join_kernel<D, 4><<<dim3(ceil_div(a.Hq, 4), a.B), 256, 0, stream>>>(
        a, parts, kTracks, tile_keys);
  } else {
    const int slices = std::clamp(1024 / heads, 1, D / 32);
    attention_join_kernel<D, 1><<<dim3(a.Hq, a.B, slices), 256, 0, stream>>>(a, parts, kTracks,
                                                                            tile_keys);
  }
  return hipGetLastError();
}

template <int D, bool kFp8, int kTracks, bool kShared>
hipError_t launch_list(const AttentionArgs& a, bool whole, hipStream_t stream) {
  return a.sel != nullptr ? launch_cfg<D, kFp8, kTracks, kShared, true>(a, whole, stream)
                          : launch_cfg<D, kFp8, kTracks, kShared, false>(a, whole, stream);
}

// Few tiles a row at most (short contexts, windows, short lists): every row is
// one workgroup's, and there is nothing to join.  Splitting and joining take
// 4 to 5 us in all, a tile of a workgroup alone 0.9, and the more rows there
// are the less a split is for.  While every row of a single track has a
// workgroup at once, its four waves take stripes of the row, else four tracks.
// 32 query heads over 8 of 128, us of (four tracks split / four tracks whole /
// stripes whole): 1 request of up to 64 tokens 8.8 / 7.5 / 5.8, of 256 9.6 / -
// / 8.0, of 512 11.3 / - / 11.0; 16 of 384 12.9 / - / 10.0; 64 of 256 18.7 /
// 19.7 / 12.1, of 768 31.6 / - / 28.7; 256 of 64 - / 12.3 / 19.7, of 512 72.6 /
// 62.7 / 65.8.  With 8 bits 64 of 512 20.0 / - / 13.9.  256-wide tiles are twice
// the bytes and have half the workgroups.
//
// Rows that wait for a workgroup to come free are striped while they are short,
// the longer the more of them there are.  Us of (four tracks split / stripes whole)
// for lengths of 1/8 to the whole of the limit, and all at it: 72 requests of 300
// 20.1 / 19.3 and 26.8 / 23.8; 65 of 768 27.0 / 36.7 and 44.3 / 48.6, 96 of 768
// 32.8 / 37.5 and 58.0 / 53.4, 104 of 640 32.0 / 32.9 and 55.5 / 47.5, 128 of 768
// 40.4 / 40.3 and 71.5 / 65.6.  256 wide, 112 of 384 25.8 / 28.7 and 39.7 / 35.5;
// 8 bits, 65 of 1000 23.1 / 30.6 and 33.5 / 36.8, 112 of 1000 31.0 / 31.3 and 51.5
// / 43.7.
template <int D, bool kFp8>
hipError_t launch_tracks(const AttentionArgs& a, hipStream_t stream) {
  using T = Tile<D, kFp8>;
  const int tracks = tracks_of(a.Hq, a.H), group = tracks_per_group(tracks);
  const long long rows = (long long)a.B * tracks, keys = most_keys(a);
  const bool whole = keys <= std::min(4 + rows / group / 16, 32ll) * T::kKeys * (4 / group);
  const long long at_once = T::kPerCu * kCus;
  auto striped = [](long long tiles) { return tiles / (3 - T::kPerCu) * T::kKeys * 4; };  // keys
  const bool waiting = rows <= 2 * at_once && keys <= striped(5 + 8 * (rows - at_once) / at_once);
  if (keys <= striped(std::min(5 + rows / 16, 12ll)) && (rows <= at_once || (!whole && waiting)))
    return launch_list<D, kFp8, 1, false>(a, true, stream);
  const bool shared = tracks > a.H;
  switch (group) {
    case 4:
      return shared ? launch_list<D, kFp8, 4, true>(a, whole, stream)
                    : launch_list<D, kFp8, 4, false>(a, whole, stream);
    case 2:
      return shared ? launch_list<D, kFp8, 2, true>(a, whole, stream)
                    : launch_list<D, kFp8, 2, false>(a, whole, stream);
    default: return launch_list<D, kFp8, 1, false>(a, whole, stream);
  }
}

}  // namespace

hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream) {
  const bool fp8 = a.dtype == kCacheFp8;
  switch (a.D) {
    case 64: return fp8 ? launch_tracks<64, true>(a, stream) : launch_tracks<64, false>(a, stream);
    case 128: return fp8 ? launch_tracks<128, true>(a, stream) : launch_tracks<128, false>(a, stream);
    case 256: return fp8 ? launch_tracks<256, true>(a, stream) : launch_tracks<256, false>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mova

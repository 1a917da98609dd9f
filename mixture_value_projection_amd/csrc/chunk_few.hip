// Chunk attention of requests with few rows (one token, drafts): up to sixteen
// rows, tokens times query heads, of a key head.
//
// Such a request does a few flops for each byte of cache, so everything serves
// the stream of keys and values, as in the attention of one token: the tiles of all
// such requests lie in one line, cut into equal stretches; a workgroup's four waves
// take four key heads at the same positions, or stripes of the tiles where there
// are fewer; each wave is a pipeline of its own, a ring of tiles in LDS filled by
// direct loads.  Sixteen rows take part in a wave's products, so a request of more
// would be read more than once.
//
// Bound by the cache's bytes: 64 requests of 500 to 8000 tokens with four new ones, 32
// heads over 8 of 128, 738 MB in 130 us, 5.7 TB/s.
//
// What differs from one token: rows see different keys, so logits are hidden row by
// row in the tiles where the request's new tokens lie (and where its windows begin),
// and a row whose sums become infinite or NaN is formed once more from the keys that
// it sees alone.
#include <algorithm>
#include <atomic>

#include "chunk.h"
#include "kernels.h"
#include "paged_tile.h"

namespace mova {

namespace {

static_assert(kFewRows == 16, "the rows of a product");
// Tiles of a stretch at least: a row of so few is not cut.  (Of two, four and eight: 1
// token after 130 12.0, 13.7 and 16.7 us, 64 requests of 32 to 256 tokens 25.4, 26.0 and
// 29.4, 1 token after 8000 30.8, 20.2 and 19.5.)
constexpr int kLeastTiles = 4;

// Request b as this kernel sees it.
template <int kTracks>
struct Few {
  Chunk c;
  int lo;      // first key that any row sees
  int rows;    // of a key head; 0: another kernel's, or none
  int n;       // tiles of the keys
  __device__ __forceinline__ long long units(int H) const { return (long long)n * (H / kTracks); }
};
template <int kTracks>
__device__ __forceinline__ Few<kTracks> few_of(const ChunkArgs& a, int b, int tile_keys) {
  Few<kTracks> f;
  f.c = chunk_of(a, b);
  f.rows = f.c.live * (a.Hq / a.H);
  if (f.rows > a.few) f.rows = 0;
  f.lo = a.window > 0 ? max(0, f.c.at + 1 - a.window) : 0;
  f.n = f.rows == 0 ? 0 : ceil_div(f.c.at + f.c.live - f.lo, tile_keys);
  return f;
}

}  // namespace

template <int D, bool kFp8, int kTracks>
__global__ __launch_bounds__(256) void chunk_few_kernel(ChunkArgs a, Parts parts, FastDiv by_block,
                                                        FastDiv by_group) {
  using T = Tile<D, kFp8>;
  constexpr int kStripes = 4 / kTracks;
  constexpr int S = T::kStages;
  constexpr int kSub = T::kKeys / 16;  // 16-key parts of a tile
  constexpr int kCols = D / 16;
  constexpr int kGroupLoads = 2 * T::kLoads + 1;
  static_assert((S - 1) * kGroupLoads < 64, "outstanding loads");
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  __shared__ Shared s_line;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int tsub = wave / kStripes, stripe = wave % kStripes;
  const int G = a.Hq / a.H;
  char* ring = lds + wave * T::kLds;
  int* pages = (int*)(ring + T::kRing);
  constexpr int kTileKeys = T::kKeys * kStripes;

  // Neighbouring stretches on one XCD.
  const int slots = gridDim.x;
  const int slot = (int)(blockIdx.x & 7) * (slots >> 3) + (int)(blockIdx.x >> 3);
  Line line;
  const bool work = chunk_line<4>(
      a.B, slot, slots, kLeastTiles,
      [&](int b) { return few_of<kTracks>(a, b, kTileKeys).units(a.H); }, s_line, &line);
  if (tid == 0) parts.split[slot].n = 0;
  clear_rows(a, tid);
  if (!work) return;

  const uint32_t row_bytes = (uint32_t)a.H * T::kRow;
  int b = line.b;
  long long first = line.first;  // first unit of request b
  Few<kTracks> f = few_of<kTracks>(a, b, kTileKeys);
  for (long long pos = line.start; pos < line.end;) {
    while (pos >= first + f.units(a.H)) {
      first += f.units(a.H);
      if (++b >= a.B) return;
      f = few_of<kTracks>(a, b, kTileKeys);
    }
    const int heads = (int)floor_div(pos - first, f.n);  // kTracks of them
    const int t0 = (int)(pos - first - (long long)heads * f.n);
    const int t1 = (int)min((long long)f.n, t0 + (line.end - pos));
    pos += t1 - t0;
    const int nt = t1 - t0;
    const bool all = nt == f.n;
    const int h = heads * kTracks + tsub;
    const int len = f.c.at + f.c.live;
    const int32_t* table = a.table + (size_t)b * a.max_blocks;
    if (t0 == 0 && !all && tid == 0) {
      Split p;
      p.row0 = (long long)f.c.row0 * a.Hq + (long long)heads * kTracks * G;
      p.before = 0;
      p.n = (int)floor_div(line.stretch - nt + f.n - 1, line.stretch) + 1;
      p.lo = 0;
      p.hi = 0;
      p.rows = f.rows;
      p.heads = 0;
      parts.split[slot] = p;
    }
    // (As in the other kernel.)
    if (t0 > 0 && t0 + nt < f.n && tid == 0)
      parts.split[slot].n = -(int)floor_div(t0 + line.stretch - 1, line.stretch);

    // The lane's row.
    const bool has_row = r16 < f.rows;
    const int token = fast_div(r16, by_group);
    const size_t row = (size_t)(f.c.row0 + token) * a.Hq + h * G + (r16 - token * G);
    const int limit = has_row ? f.c.at + token : 0x3fffffff;
    const int lower = has_row && a.window > 0 ? max(0, limit + 1 - a.window) : 0;
    // Keys from `shared` up to `own` are seen by all rows here.
    const int own = f.c.at + 1;
    const int shared = a.window > 0 ? max(0, f.c.at + f.c.live - a.window) : 0;

    auto key_of = [&](int x) { return f.lo + ((t0 + x) * kStripes + stripe) * T::kKeys; };
    auto table_address = [&](int x) {
      const int p = key_of(x) + (lane & (T::kKeys - 1));
      return table + min(fast_div(p, by_block), a.max_blocks - 1);
    };
    // Issues tile x: the loads of its keys and values, addressed by its block
    // numbers, and the fetch of those of tile x + S.  Returns which of its keys are
    // there (bit = key).
    auto issue = [&](int x, int page) -> uint32_t {
      const int p = key_of(x) + (lane & (T::kKeys - 1));
      const bool ok = p < len && page >= 0 && page < a.num_blocks;
      const uint32_t mask = (uint32_t)__ballot(ok) & (uint32_t)((1ull << T::kKeys) - 1);
      const int slot_of = ok ? page * a.block_size + (p - fast_div(p, by_block) * a.block_size) : 0;
      char* stage = ring + (x & (S - 1)) * 2 * T::kSide;
      uint32_t row_slot[T::kLoads];  // exchanged together, before the first load
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i)
        row_slot[i] = (uint32_t)__shfl(slot_of, i * T::kRowsPerLoad + lane / T::kChunks);
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) {
        const int rr = i * T::kRowsPerLoad + lane / T::kChunks;
        const size_t off = (size_t)row_slot[i] * row_bytes + (size_t)h * T::kRow;
        const int c = lane % T::kChunks;
        piece_to_lds<T::kStream>((const char*)a.k_cache + off + (c ^ T::swizzle_k(rr)) * 16,
                                 stage + i * 1024);
        piece_to_lds<T::kStream>((const char*)a.v_cache + off + (c ^ T::swizzle_v(rr)) * 16,
                                 stage + T::kSide + i * 1024);
      }
      word_to_lds(table_address(x + S), pages + (x & (S - 1)) * 64);
      return mask;
    };

    // Queries: with 8-bit keys a lane's 16-byte piece serves two products.
    Frag16 qf[D / 32];
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int d = kFp8 ? 64 * (u / 2) + 16 * g4 + 8 * (u & 1) : 32 * u + 8 * g4;
      qf[u].u = u32x4{0u, 0u, 0u, 0u};
      if (has_row) qf[u].u = load16(a.q + row * D + d);
    }
    const float ks = a.k_scale != nullptr ? a.k_scale[h] : 1.f;
    const float vs = a.v_scale != nullptr ? a.v_scale[h] : 1.f;
    const float qs = a.scale * ks * kLog2e;  // logits in powers of two

    uint32_t masks[S] = {};  // of the tiles in the ring
    // The last segment's LDS reads are done before the ring is filled again.
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < S; ++i) word_to_lds(table_address(i), pages + i * 64);
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
      // Tile x and the fetch issued with it have landed.
      if (x >= 0) wait_groups<S - 1, kGroupLoads>(min(S - 1, nt - 1 - x));
      asm volatile("" ::: "memory");
      char* stage = ring + (x & (S - 1)) * 2 * T::kSide;
      constexpr uint32_t kAll = (uint32_t)((1ull << T::kKeys) - 1);
      if (x >= 0 && mask != 0) {
        if (mask != kAll) {
          // Values that are not there become zeros: their weight is zero, but what
          // lies there may be infinite or NaN.
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
        const int base = key_of(x);
        if (mask != kAll || base + T::kKeys > own || base < shared) {
          const uint32_t of_lane = mask >> (4 * g4);
          const int above = limit - base - 4 * g4, below = lower - base - 4 * g4;
#pragma unroll
          for (int t = 0; t < kSub; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((of_lane >> (16 * t + i)) & 1) || 16 * t + i > above || 16 * t + i < below)
                p[t][i] = -__builtin_huge_valf();
        }
#pragma unroll
        for (int t = 0; t < kSub; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, p[t][i]);
        top = max_over_groups(top);
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
            high.e[4 * t + i] = (bf16_t)e;
            low.e[4 * t + i] = (bf16_t)(e - (float)high.e[4 * t + i]);
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
        // Tile x + S takes this tile's place; its block numbers came with tile x.
        const int page = pages[(x & (S - 1)) * 64 + lane];
        __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
        asm volatile("" ::: "memory");
        masks[S - 1] = issue(x + S, page);
      }
    }

    // The four lanes of a row hold its sum in parts.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
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
    float largest = 0.f;  // NaN counts as the largest
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) largest = __builtin_elementwise_maximum(largest, fabsf(o[c][i]));
    const bool odd = has_row && l > 0.f && l < __builtin_huge_valf() &&
                     !(largest < __builtin_huge_valf());
    uint64_t odd_lanes = __ballot(odd);
    odd_lanes |= odd_lanes >> 32;
    const uint32_t again = (uint32_t)(odd_lanes | odd_lanes >> 16) & 0xffffu;
    auto sink_of = [&](size_t at, int lane_row) {
      Sink<D> to;
      to.out = all ? a.out + at * D : nullptr;
      to.lse = a.lse != nullptr ? a.lse + at : nullptr;
      const size_t part =
          ((size_t)(slot * 2 + (t0 == 0 ? 1 : 0)) * kTracks + tsub) * 16 + lane_row;
      to.o = parts.o + part * D;
      to.ml = parts.ml + part * 2;
      return to;
    };
    const float scale = l == 0.f ? 0.f : vs / l;
    if (has_row) {
      const Sink<D> to = sink_of(row, r16);
      if (!((again >> r16) & 1)) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const f32x4 y = {o[c][0] * scale, o[c][1] * scale, o[c][2] * scale, o[c][3] * scale};
          if (all) {
            uint2 w;
            w.x = (uint32_t)f32_to_bf16_bits(y[0]) | ((uint32_t)f32_to_bf16_bits(y[1]) << 16);
            w.y = (uint32_t)f32_to_bf16_bits(y[2]) | ((uint32_t)f32_to_bf16_bits(y[3]) << 16);
            *reinterpret_cast<uint2*>(to.out + 16 * c + 4 * g4) = w;
          } else {
            *reinterpret_cast<f32x4*>(to.o + 16 * c + 4 * g4) = y;
          }
        }
      }
      if (g4 == 0) to.put_sum(l == 0.f ? -__builtin_huge_valf() : m, l);
    }
    if (__builtin_expect(again != 0, 0)) {
      // (Lanes i and i + 32 have row i % 32 there, so i % 16 where it is one of these.)
      const bool mine = (lane & 16) == 0 && ((again >> r16) & 1);
      attend_again<D, kFp8>(a, by_block, b, h, mine ? a.q + row * D : nullptr, qs, m,
                            mine ? limit : -1, lower, f.lo + t0 * kTileKeys,
                            min(len, f.lo + t1 * kTileKeys), 0, D / 32, scale,
                            [&](int channel, float y) {
                              if (mine) sink_of(row, r16).put1(channel, y);
                            });
    }
  }
}

namespace {

size_t part_rows(int groups, int H) { return (size_t)groups * 2 * chunk_few_tracks(H) * 16; }

template <int D, bool kFp8, int kTracks>
hipError_t launch_cfg(const ChunkArgs& a, const Parts& parts, int groups, hipStream_t stream) {
  using T = Tile<D, kFp8>;
  static std::atomic<unsigned long long> done{0};
  hipError_t e = once_per_device(done, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(chunk_few_kernel<D, kFp8, kTracks>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, 4 * T::kLds);
  });
  if (e != hipSuccess) return e;
  chunk_few_kernel<D, kFp8, kTracks><<<groups, 256, 4 * T::kLds, stream>>>(
      a, parts, make_fast_div(a.block_size), make_fast_div(a.Hq / a.H));
  return hipGetLastError();
}

template <int D, bool kFp8>
hipError_t launch_tracks(const ChunkArgs& a, const Parts& parts, int groups, hipStream_t stream) {
  switch (chunk_few_tracks(a.H)) {
    case 4: return launch_cfg<D, kFp8, 4>(a, parts, groups, stream);
    case 2: return launch_cfg<D, kFp8, 2>(a, parts, groups, stream);
    default: return launch_cfg<D, kFp8, 1>(a, parts, groups, stream);
  }
}

// Workgroups where the keys are many, and the line's units: both types of pool are taken
// for the one with more, as the scratch's size is asked for without the type.
template <int D>
int groups_of(int B, int H, long long most) {
  static_assert(Tile<D, true>::kPerCu == Tile<D, false>::kPerCu, "a size for both types");
  constexpr int kKeys = std::min(Tile<D, true>::kKeys, Tile<D, false>::kKeys);
  const int tracks = chunk_few_tracks(H);
  const double tiles = (double)((most + kKeys - 1) / kKeys);  // a stripe's are at most as many
  return groups_for(tiles * B * (H / tracks), kLeastTiles, kCus * Tile<D, true>::kPerCu);
}

}  // namespace

int chunk_few_groups(int T, int B, int H, int D, long long most) {
  const int requests = std::min(T, B);  // that have a token
  return D == 64    ? groups_of<64>(requests, H, most)
         : D == 128 ? groups_of<128>(requests, H, most)
                    : groups_of<256>(requests, H, most);
}

int chunk_few_tracks(int H) { return H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1; }

size_t chunk_few_floats(int groups, int H, int D) {
  return split_floats(groups) + part_rows(groups, H) * (2 + D);
}

Parts chunk_few_parts(float* scratch, int groups, int H) {
  Parts parts;
  parts.split = (Split*)scratch;
  parts.ml = scratch + split_floats(groups);
  parts.o = parts.ml + part_rows(groups, H) * 2;
  return parts;
}

hipError_t launch_chunk_few(const ChunkArgs& a, const Parts& parts, int groups,
                            hipStream_t stream) {
  const bool fp8 = a.dtype == kCacheFp8;
  switch (a.D) {
    case 64:
      return fp8 ? launch_tracks<64, true>(a, parts, groups, stream)
                 : launch_tracks<64, false>(a, parts, groups, stream);
    case 128:
      return fp8 ? launch_tracks<128, true>(a, parts, groups, stream)
                 : launch_tracks<128, false>(a, parts, groups, stream);
    case 256:
      return fp8 ? launch_tracks<256, true>(a, parts, groups, stream)
                 : launch_tracks<256, false>(a, parts, groups, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mova

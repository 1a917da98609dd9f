// What the kernels that stream a request's keys and values past a few rows of
// queries share: the tiles of a wave's ring and the reads from them.
#pragma once

#include <type_traits>

#include "paged.h"

namespace mova {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2;

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

}  // namespace mova

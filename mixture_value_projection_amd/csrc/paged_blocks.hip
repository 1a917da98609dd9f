// Upkeep of the paged cache's blocks: contents copied, rows of the block table
// forked and given back, and blocks moved to the low end of the pool.
//
// A block that several rows of the table hold has a share count, the number of
// its holders beyond the first.  A free block, and one with a single holder,
// has 0, so that the plan, which hands out and takes back whole blocks, needs
// to know nothing of it.
//
// All of these move a few bytes a block (the copy apart), so they cost their
// latency: few launches, and as few memory round trips in a row as the result
// allows.  What depends on an order is brought to one that no execution
// changes: pairs by their index, blocks by their number.
#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "paged.h"

namespace mova {

namespace {

constexpr int kForkThreads = 256;
constexpr int kFreeThreads = 1024;
constexpr int kFreeAtOnce = 8;
constexpr int kFreeRows = kMaxRequests / kFreeThreads;  // of a thread

constexpr int kRankWords = kRankBlocks / 32;

__device__ __forceinline__ bool in_pool(int page, int num_blocks) {
  return page >= 0 && page < num_blocks;
}

// Length of a row, kept inside it.
__device__ __forceinline__ int clamp_len(int n, int most) { return min(max(n, 0), most); }

}  // namespace

// ---- copy ---------------------------------------------------------------------

// Workgroup items: 16 KB of a block's keys, values and bounds, seen as one run of
// pieces; a thread has four pieces in flight, and every item has a workgroup of its
// own, as far as a grid goes (770 MB read and written in blocks of 32 KB: 2048
// workgroups with items in turn 180 us, this 150).  Pools larger than the last cache
// pass the caches by: that takes 132 us (5.8 TB/s) for those 770 MB, but for 60 MB of
// a pool of 119 MB 14 us, and 11 through the caches.  (The host knows the pool, not how
// many of the pairs are there.  Copied again and again in pools of 2 GB, so that what fits
// stays in the caches: 2 MB 5.3 past and 4.9 through them, 121 MB 26.7 and 22.3, 393 MB 81
// and 83, 1573 MB 309 and 326.)
constexpr size_t kLastCache = (size_t)256 << 20;
constexpr int kCopyGrid = 65536;
constexpr int kCopyAtOnce = 4, kCopyPieces = 256 * kCopyAtOnce;

template <bool kPast>
__global__ __launch_bounds__(256) void paged_copy_kernel(CopyArgs a) {
  const int count = a.count == nullptr ? a.n : min(max(*a.count, 0), a.n);
  const int pieces = a.pieces[0] + a.pieces[1] + a.pieces[2];
  const int parts = ceil_div(pieces, kCopyPieces);
  const long long items = (long long)count * parts;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int pair = (int)floor_div(item, parts);
    const int first = (int)(item - (long long)pair * parts) * kCopyPieces + (int)threadIdx.x;
    const int src = a.src[pair], dst = a.dst[pair];
    if (!in_pool(src, a.num_blocks) || !in_pool(dst, a.num_blocks) || src == dst) continue;
    u32x4 x[kCopyAtOnce];
    u32x4* to[kCopyAtOnce];
#pragma unroll
    for (int i = 0; i < kCopyAtOnce; ++i) {
      int p = first + 256 * i;
      to[i] = nullptr;
      if (p >= pieces) continue;
      u32x4* pool = a.pool[0];
      int width = a.pieces[0];
      if (p >= width) {
        p -= width;
        pool = a.pool[1];
        width = a.pieces[1];
        if (p >= width) {
          p -= width;
          pool = a.pool[2];
          width = a.pieces[2];
        }
      }
      const u32x4* from = pool + (size_t)src * width + p;
      x[i] = kPast ? __builtin_nontemporal_load(from) : *from;
      to[i] = pool + (size_t)dst * width + p;
    }
#pragma unroll
    for (int i = 0; i < kCopyAtOnce; ++i)
      if (to[i] != nullptr) {
        if constexpr (kPast)
          __builtin_nontemporal_store(x[i], to[i]);
        else
          *to[i] = x[i];
      }
  }
}

hipError_t launch_paged_copy(const CopyArgs& a, hipStream_t stream) {
  const long long parts = ceil_div(a.pieces[0] + a.pieces[1] + a.pieces[2], kCopyPieces);
  const int grid = (int)std::min<long long>(a.n * parts, kCopyGrid);
  const size_t bytes = (size_t)a.num_blocks * (a.pieces[0] + a.pieces[1] + a.pieces[2]) * 16;
  if (bytes > kLastCache)
    paged_copy_kernel<true><<<grid, 256, 0, stream>>>(a);
  else
    paged_copy_kernel<false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

// ---- fork ---------------------------------------------------------------------

// Every workgroup reads all pairs and forms the running sum of the blocks that
// they take; then it goes through its share of their entries.  Parents' rows
// are only read and children's only written, so no workgroup waits for another.
// Bound by its round trips: lengths, then entries, then counts.  56 rows of up to 500
// blocks 4.6 us, 12 of up to 6250 4.8.
__global__ __launch_bounds__(kForkThreads) void paged_fork_kernel(ForkArgs a, FastDiv by_block,
                                                                  int chunks) {
  extern __shared__ int fork_lds[];
  int* s_owner = fork_lds;      // [B] the pair whose child the row is
  int* s_parent = s_owner + a.B;  // [B] whether it is a parent
  int* s_row = s_parent + a.B;  // [n] parent's row, -1: the pair gets nothing
  int* s_len = s_row + a.n;     // [n] tokens taken over
  int* s_upto = s_len + a.n;    // [n] blocks taken up to and with it
  __shared__ long long tmp[kForkThreads / 64];
  const int tid = threadIdx.x, bs = a.block_size;
  const int most = a.max_blocks * bs;
  const int have = min(max(*a.free_count, 0), a.free_capacity);
  for (int b = tid; b < a.B; b += kForkThreads) {
    s_owner[b] = a.n;
    s_parent[b] = 0;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kForkThreads) {
    const int p = a.parents[i], c = a.children[i];
    const bool ok = p >= 0 && p < a.B && c >= 0 && c < a.B && p != c;
    s_row[i] = ok ? p : -1;
    s_len[i] = ok ? c : -1;  // for now
    if (ok) {
      atomicMin(&s_owner[c], i);
      s_parent[p] = 1;
    }
  }
  __syncthreads();
  const int per = ceil_div(a.n, kForkThreads);
  const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
  long long need = 0, total;
  for (int i = i0; i < i1; ++i) {
    const int p = s_row[i], c = s_len[i];
    const bool ok = p >= 0 && s_owner[c] == i && !s_parent[c];
    int len = 0;
    if (ok) {
      len = clamp_len(a.cached[p], most);
      if (a.take != nullptr) len = clamp_len(a.take[i], len);
    }
    s_row[i] = ok ? p : -1;
    s_len[i] = len;
    need += ok && len != fast_div(len, by_block) * bs;
  }
  int upto = (int)block_exclusive_scan<kForkThreads / 64>(need, tmp, &total);
  for (int i = i0; i < i1; ++i) {
    const int len = s_len[i];
    const bool part = s_row[i] >= 0 && len != fast_div(len, by_block) * bs;
    upto += part;
    if (part && upto > have) s_row[i] = -1;
    s_upto[i] = upto;
  }
  __syncthreads();

  if (blockIdx.x == 0) {
    if (tid == 0) *a.free_count_out = have - (int)min(total, (long long)have);
    for (int b = tid; b < a.B; b += kForkThreads) {
      const int i = s_owner[b];
      const bool child = i < a.n && s_row[i] >= 0;
      a.seq_lens[b] = child ? s_len[i] : clamp_len(a.cached[b], most);
    }
    for (int i = tid; i < a.n; i += kForkThreads) {
      const int p = s_row[i], len = s_len[i], full = fast_div(len, by_block);
      int src = -1, dst = -1;
      if (p >= 0 && len != full * bs) {
        dst = a.free_blocks[have - s_upto[i]];
        src = a.table[(size_t)p * a.max_blocks + full];
        a.table[(size_t)a.children[i] * a.max_blocks + full] = dst;
      }
      a.copy_src[i] = src;
      a.copy_dst[i] = dst;
    }
  }
  // Items: a pair's full blocks, every chunks-th run of 256 of them.
  const int items = a.n * chunks;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int chunk = item / a.n, i = item - chunk * a.n;
    if (s_row[i] < 0) continue;
    const int full = fast_div(s_len[i], by_block);
    const int32_t* from = a.table + (size_t)s_row[i] * a.max_blocks;
    int32_t* to = a.table + (size_t)a.children[i] * a.max_blocks;
    for (long long j = chunk * kForkThreads + tid; j < full; j += chunks * kForkThreads) {
      const int page = from[j];
      to[j] = page;
      if (in_pool(page, a.num_blocks)) atomicAdd(&a.shares[page], 1);
    }
  }
}

hipError_t launch_paged_fork(const ForkArgs& a, hipStream_t stream) {
  if (a.B > kMaxRequests || a.n > kMaxRequests) return hipErrorInvalidValue;
  const int chunks = std::min(ceil_div(a.max_blocks, kForkThreads),
                              std::max(1, 512 / std::max(a.n, 1)));
  const int grid = std::min(std::max(a.n * chunks, 1), 512);
  paged_fork_kernel<<<grid, kForkThreads, (size_t)(2 * a.B + 3 * a.n) * 4, stream>>>(
      a, make_fast_div(a.block_size), chunks);
  return hipGetLastError();
}

// ---- free ---------------------------------------------------------------------

// The pool lies in runs of free_run() blocks, a workgroup each.  The first kernel
// finds out which rows are cut where, every workgroup for itself and from the counts
// as they came; it goes through all entries that are given back and counts, in LDS,
// those of its blocks.  What it leaves is how often each block is let go, and how many
// of a run's blocks are let go more often than they have holders beyond the first.
// With those numbers the second one brings the counts down and puts the blocks on
// the stack, highest first.
//
// A workgroup alone waits for memory at each turn: the 28,689 entries that 203 rows
// give back took one 80 us with atomics on the counts and 32 with counts in LDS; these
// two take 17 and 4.  The 1051 of a step of 64 rows took it 8; 6 and 4.  As each workgroup
// reads all entries, the time grows with them: 262,144 129 us for both, 1,048,576 470, a
// sixteenth of those 45.
__global__ __launch_bounds__(kFreeThreads) void free_count_kernel(FreeArgs a, FastDiv by_block,
                                                                  int run) {
  extern __shared__ __attribute__((aligned(16))) char free_lds[];
  // Rows that give back: entries given back before the row, and its first one's
  // place in the table less that.
  long long* s_first = (long long*)free_lds;     // [B]
  long long* s_base = s_first + a.B;             // [B]
  uint32_t* s_gone = (uint32_t*)(s_base + a.B);  // [run / 2] two blocks' counts a word
  __shared__ long long tmp[3][kFreeThreads / 64];
  const int tid = threadIdx.x, bs = a.block_size;
  const int most = a.max_blocks * bs;
  const int lo = blockIdx.x * run, here = min(run, a.num_blocks - lo);
  auto blocks = [&](int n) { return fast_div(n + bs - 1, by_block); };
  auto kept = [&](int b, int n) {
    const int m = clamp_len(a.keep[b], n), full = fast_div(m, by_block);
    if (m == n || m == full * bs) return m;
    const int page = a.table[(size_t)b * a.max_blocks + full];
    return in_pool(page, a.num_blocks) && a.shares[page] > 0 ? n : m;
  };
  for (int w = tid; w < run / 2; w += kFreeThreads) s_gone[w] = 0;

  const int per = ceil_div(a.B, kFreeThreads);
  long long gone = 0, all_gone, giving = 0, rows;
  int going[kFreeRows];
  long long base[kFreeRows];
#pragma unroll
  for (int i = 0; i < kFreeRows; ++i) {
    const int b = tid * per + i;
    going[i] = 0;
    if (i >= per || b >= a.B) continue;
    const int n = clamp_len(a.cached[b], most), m = kept(b, n);
    if (blockIdx.x == 0) a.seq_lens[b] = m;
    going[i] = blocks(n) - blocks(m);
    base[i] = (long long)b * a.max_blocks + blocks(m);
    gone += going[i];
    giving += going[i] > 0;
  }
  long long first = block_exclusive_scan<kFreeThreads / 64>(gone, tmp[0], &all_gone);
  long long row = block_exclusive_scan<kFreeThreads / 64>(giving, tmp[1], &rows);
#pragma unroll
  for (int i = 0; i < kFreeRows; ++i) {
    if (going[i] == 0) continue;
    s_first[row] = first;
    s_base[row++] = base[i] - first;
    first += going[i];
  }
  __syncthreads();
  // Eight entries of a thread: their pages are asked for together.
  for (long long e0 = (long long)tid * kFreeAtOnce; e0 < all_gone;
       e0 += kFreeThreads * kFreeAtOnce) {
    int r = last_at_most(s_first, (int)rows, e0);
    long long from = s_base[r], next = r + 1 < rows ? s_first[r + 1] : all_gone;
    int page[kFreeAtOnce];
#pragma unroll
    for (int i = 0; i < kFreeAtOnce; ++i) {
      const long long e = min(e0 + i, all_gone - 1);
      if (e == next) {
        from = s_base[++r];
        next = r + 1 < rows ? s_first[r + 1] : all_gone;
      }
      page[i] = a.table[from + e];
    }
#pragma unroll
    for (int i = 0; i < kFreeAtOnce; ++i) {
      const uint32_t p = (uint32_t)(page[i] - lo);
      if (e0 + i < all_gone && page[i] >= lo && p < (uint32_t)here)
        atomicAdd(&s_gone[p >> 1], 1u << 16 * (p & 1));
    }
  }
  __syncthreads();
  int last = 0;
  for (int w = tid; w < ceil_div(here, 2); w += kFreeThreads) {
    const uint32_t n = s_gone[w];
    a.scratch[kFreeRuns + lo / 2 + w] = n;
    if (n == 0) continue;
    last += (int)(n & 0xffffu) > max(a.shares[lo + 2 * w], 0);
    last += (int)(n >> 16) > max(a.shares[lo + min(2 * w + 1, here - 1)], 0);
  }
  long long all;
  block_exclusive_scan<kFreeThreads / 64>(last, tmp[2], &all);
  if (tid == 0) a.scratch[blockIdx.x] = (uint32_t)all;
}

__global__ __launch_bounds__(256) void free_apply_kernel(FreeArgs a, int run) {
  static_assert(kFreeRuns == 256, "a thread a run");
  __shared__ long long tmp[2][4];
  __shared__ int s_mine[4];
  __shared__ uint32_t s_last[kMaxUpkeepBlocks / kFreeRuns / 2];  // a word's blocks that go
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * run, here = min(run, a.num_blocks - lo);
  const int count = min(max(*a.free_count, 0), a.free_capacity);
  const int at = tid < (int)gridDim.x ? (int)a.scratch[tid] : 0;
  long long above, all;
  block_exclusive_scan<4>(tid > (int)blockIdx.x ? at : 0, tmp[0], &above);
  block_exclusive_scan<4>(at, tmp[1], &all);
  if (blockIdx.x == 0 && tid == 0)
    *a.free_count_out = (int)min(count + all, (long long)a.free_capacity);

  // A wave's words, highest first, a lane a word.
  const int words = ceil_div(here, 2), mine = run / 8;
  const int top = words - wave * mine, bottom = max(top - mine, 0);
  int pushed = 0;
  for (int w0 = top; w0 > bottom; w0 -= 64) {
    const int w = w0 - 1 - lane;
    uint32_t last = 0;
    if (w >= bottom) {
      const uint32_t n = a.scratch[kFreeRuns + lo / 2 + w];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int times = (int)(n >> 16 * i & 0xffffu);
        if (times == 0) continue;
        const int held = max(a.shares[lo + 2 * w + i], 0);
        a.shares[lo + 2 * w + i] = max(held - times, 0);
        last |= (uint32_t)(times > held) << i;
      }
      s_last[w] = last;
    }
    pushed += __popcll(__ballot(last & 1)) + __popcll(__ballot(last & 2));
  }
  if (lane == 0) s_mine[wave] = pushed;
  __syncthreads();
  long long to = count + above;
  for (int w = 0; w < wave; ++w) to += s_mine[w];
  for (int w0 = top; w0 > bottom && pushed > 0; w0 -= 64) {
    const int w = w0 - 1 - lane;
    const uint32_t last = w >= bottom ? s_last[w] : 0;
    const uint64_t odd = __ballot(last & 2), even = __ballot(last & 1);
    const uint64_t before = (1ull << lane) - 1;
    const long long mark = to + __popcll(odd & before) + __popcll(even & before);
    const long long after = mark + (last >> 1);
    if ((last & 2) && mark < a.free_capacity) a.free_blocks[mark] = lo + 2 * w + 1;
    if ((last & 1) && after < a.free_capacity) a.free_blocks[after] = lo + 2 * w;
    to += __popcll(odd) + __popcll(even);
  }
}

hipError_t launch_paged_free(const FreeArgs& a, hipStream_t stream) {
  if (a.B > kMaxRequests || a.num_blocks > kMaxUpkeepBlocks) return hipErrorInvalidValue;
  const int run = free_run(a.num_blocks), runs = std::max(ceil_div(a.num_blocks, run), 1);
  free_count_kernel<<<runs, kFreeThreads, (size_t)a.B * 16 + run * 2, stream>>>(
      a, make_fast_div(a.block_size), run);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  free_apply_kernel<<<runs, 256, 0, stream>>>(a, run);
  return hipGetLastError();
}

// ---- compaction ---------------------------------------------------------------

// With L blocks in use and the edge at max(limit, L), the i-th used block at or
// above the edge goes to the i-th free block below it.  There are as many free
// ones: below the edge lie edge - x of them, x the used ones there, and L - x
// used ones lie above.  Afterwards everything from the edge on is free.
//
// The first kernel, one workgroup, turns the stack into bits and counts them by
// runs of 256 blocks; with those counts in LDS, the second one ranks any block
// in a step and finds the block of any rank in a search, so that table, stack,
// counts and lists are written side by side.  Both are bound by their round trips: a
// pool of 24,274 blocks, 9000 and more of them free, 4.8 and 7.1 us, one of 1752 2.8 and
// 5.9.  Of larger ones, half free, the first takes most: 262,144 blocks 36 us for both,
// 1,048,576 217.
__global__ __launch_bounds__(kFreeThreads) void compact_rank_kernel(CompactArgs a) {
  extern __shared__ uint32_t compact_bits[];
  __shared__ long long tmp[kFreeThreads / 64];
  const int tid = threadIdx.x, nb = a.num_blocks;
  const int groups = compact_groups(nb);
  const int count = min(max(*a.free_count, 0), a.free_capacity);
  for (int w = tid; w < groups * kRankWords; w += kFreeThreads) compact_bits[w] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < count; i += kFreeThreads) {
    const int page = a.free_blocks[i];
    if (in_pool(page, nb)) atomicOr(&compact_bits[page >> 5], 1u << (page & 31));
  }
  __syncthreads();
  const int per = ceil_div(groups, kFreeThreads);
  const int g0 = min(tid * per, groups), g1 = min(g0 + per, groups);
  long long mine = 0, all;
  for (int w = g0 * kRankWords; w < g1 * kRankWords; ++w) mine += __popc(compact_bits[w]);
  int at = (int)block_exclusive_scan<kFreeThreads / 64>(mine, tmp, &all);
  for (int g = g0; g < g1; ++g) {
    a.scratch[g] = at;
    for (int w = 0; w < kRankWords; ++w) at += __popc(compact_bits[g * kRankWords + w]);
  }
  if (tid == 0) a.scratch[groups] = (uint32_t)all;
  for (int w = tid; w < groups * kRankWords; w += kFreeThreads)
    a.scratch[groups + 1 + w] = compact_bits[w];
}

__global__ __launch_bounds__(256) void compact_apply_kernel(CompactArgs a, FastDiv by_block) {
  extern __shared__ int s_before[];  // free blocks before each group, and all
  const int tid = threadIdx.x, nb = a.num_blocks;
  const int groups = compact_groups(nb);
  for (int g = tid; g <= groups; g += 256) s_before[g] = (int)a.scratch[g];
  __syncthreads();
  const uint32_t* bits = a.scratch + groups + 1;
  const int all = s_before[groups], used = nb - all;
  const int edge = min(max(a.limit, used), nb);
  // Free blocks before p (p <= nb), and whether p is one.
  auto rank = [&](int p, bool* is_free) -> int {
    const int g = p / kRankBlocks, w = p >> 5;
    if (g >= groups) {
      *is_free = false;
      return all;
    }
    int r = s_before[g];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kRankWords; ++i) {
      const uint32_t x = bits[g * kRankWords + i];
      if (g * kRankWords + i < w) r += __popc(x);
      if (g * kRankWords + i == w) mine = x;
    }
    *is_free = (mine >> (p & 31)) & 1;
    return r + __popc(mine & ((1u << (p & 31)) - 1));
  };
  // The free block of rank r.
  auto select = [&](int r) {
    const int g = last_at_most(s_before, groups, r);
    r -= s_before[g];
    uint32_t x = 0;
    int w = 0, at = 0;
#pragma unroll
    for (int i = 0; i < kRankWords; ++i) {
      const uint32_t y = bits[g * kRankWords + i];
      const int n = __popc(y);
      if (r >= 0 && r < n) {
        x = y;
        w = g * kRankWords + i;
        at = r;
      }
      r -= n;
    }
    for (; at > 0; --at) x &= x - 1;
    return w * 32 + __ffs((int)x) - 1;
  };
  bool edge_free;
  const int below = rank(edge, &edge_free);       // free blocks below the edge
  const int first = edge - below;                 // used ones there
  const int moves = used - first;
  // Where a block goes: -1 for a free one.
  auto target = [&](int p) {
    bool is_free;
    const int r = rank(p, &is_free);
    if (is_free) return -1;
    return p < edge ? p : select(p - r - first);
  };

  const int step = gridDim.x * 256, start = blockIdx.x * 256 + tid;
  for (int p = start; p < nb; p += step) {
    bool is_free;
    const int r = rank(p, &is_free);
    if (is_free) {
      a.remap[p] = -1;
      if (p < edge && r < moves) continue;  // taken; its count comes with the block
      a.shares_out[p] = 0;
      const int at = p < edge ? nb - edge + (below - 1 - r) : nb - 1 - p;
      if (at < a.free_capacity) a.free_out[at] = p;
      continue;
    }
    const int held = a.shares[p];
    if (p < edge) {
      a.remap[p] = p;
      a.shares_out[p] = held;
      continue;
    }
    const int i = p - r - first;
    const int to = select(i);
    a.remap[p] = to;
    a.shares_out[to] = held;
    a.shares_out[p] = 0;
    a.move_src[i] = p;
    a.move_dst[i] = to;
    if (nb - 1 - p < a.free_capacity) a.free_out[nb - 1 - p] = p;
  }
  for (int i = moves + start; i < nb / 2; i += step) {
    a.move_src[i] = -1;
    a.move_dst[i] = -1;
  }
  if (a.free_out != a.free_blocks)
    for (int i = all + start; i < a.free_capacity; i += step) a.free_out[i] = a.free_blocks[i];
  if (start == 0) {
    *a.move_count = moves;
    *a.free_count_out = min(all, a.free_capacity);
  }
  const bool apart = a.table_out != a.table;
  const int most = a.max_blocks * a.block_size;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int n = fast_div(clamp_len(a.lens[b], most) + a.block_size - 1, by_block);
    const size_t row = (size_t)b * a.max_blocks;
    for (int j = tid; j < (apart ? a.max_blocks : n); j += 256) {
      int page = a.table[row + j];
      if (j < n && in_pool(page, nb)) page = target(page);
      a.table_out[row + j] = page;
    }
  }
}

hipError_t launch_paged_compact(const CompactArgs& a, hipStream_t stream) {
  if (a.B > kMaxRequests || a.num_blocks > kMaxUpkeepBlocks) return hipErrorInvalidValue;
  static std::atomic<unsigned long long> done{0};
  hipError_t e = once_per_device(done, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(compact_rank_kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, kMaxUpkeepBlocks / 8);
  });
  if (e != hipSuccess) return e;
  const int groups = compact_groups(a.num_blocks);
  compact_rank_kernel<<<1, kFreeThreads, (size_t)groups * (kRankBlocks / 8), stream>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int grid = std::min(std::max({ceil_div(a.num_blocks, 256), a.B, 1}), 512);
  compact_apply_kernel<<<grid, 256, (size_t)(groups + 1) * 4, stream>>>(
      a, make_fast_div(a.block_size));
  return hipGetLastError();
}

}  // namespace mova

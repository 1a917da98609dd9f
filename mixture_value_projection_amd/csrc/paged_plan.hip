// Block tables and slot maps of one step, built on the GPU from the requests'
// lengths: which cache blocks each request's new tokens go to, and the slot of
// every token's row in the pools (page "IFM K2 Horizon Deep Dive: Inside
// Mixture-of-Value Attention (MoVA) ...", section "The Two Architectural
// Caching Strategies for MoVA", Option A: the routed vectors live in ordinary
// paged-attention pools).
//
// With c_b tokens stored and n_b new ones, request b holds ceil(c_b / s)
// blocks of s rows and needs ceil((c_b + n_b) / s).  Blocks come off a stack of
// free ones: the i-th block handed out by the call is entry have - 1 - i, where
// have counts the free blocks after those of ended requests (n_b < 0) were
// pushed.  A request is admitted when it needs no block, or when the running
// sum of the needs, its own included, is within have; that makes admission,
// tables and slots functions of prefix sums over the requests, with no order
// of execution in them.
//
// A few kilobytes are read and 12 bytes a token written, so the call costs its
// latency: one launch.  Every workgroup forms the prefix sums of all requests
// itself (they fit LDS) and then takes its share of the tokens, of the blocks
// handed out and of the blocks given back.  No workgroup reads what another
// writes: a token whose block is new takes it from the stack rather than from
// the table, and a block given back in this call is read from its owner's
// table row rather than from the stack.
#include <algorithm>

#include "paged.h"

namespace mova {

namespace {

constexpr int kPlanThreads = 256;

__device__ __forceinline__ int clamp_int(long long v) {
  return (int)min(v, (long long)0x7fffffff);
}

}  // namespace

__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(PlanArgs a,
                                                                  FastDiv by_block) {
  // Per request: first token row, blocks handed out before it, blocks given
  // back before it, and its stored length (-1: it gets no slots).
  extern __shared__ int plan_lds[];
  int* s_row = plan_lds;
  int* s_need = s_row + a.B;
  int* s_back = s_need + a.B;
  int* s_len = s_back + a.B;
  __shared__ long long tmp[4][kPlanThreads / 64];

  const int tid = threadIdx.x;
  const int bs = a.block_size;
  const int most = a.max_blocks * bs;  // at most 2^30
  // Blocks that n <= most tokens fill.
  auto blocks = [&](int n) { return fast_div(n + bs - 1, by_block); };
  const int per = ceil_div(a.B, kPlanThreads);
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const int count = min(max(*a.free_count, 0), a.free_capacity);

  // The thread's first request stays in registers (up to 256 requests it is the
  // only one).
  const int fresh0 = b0 < b1 ? a.fresh[b0] : 0, cached0 = b0 < b1 ? a.cached[b0] : 0;
  auto fresh = [&](int b) { return b == b0 ? fresh0 : a.fresh[b]; };
  auto cached = [&](int b) {
    return min(max(b == b0 ? cached0 : a.cached[b], 0), most);
  };

  long long rows = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = fresh(b);
    if (n >= 0) rows += n;
    else back += blocks(cached(b));
  }
  long long all_rows, all_back, all_need;
  const long long row0 = block_exclusive_scan<kPlanThreads / 64>(rows, tmp[0], &all_rows);
  const long long back0 = block_exclusive_scan<kPlanThreads / 64>(back, tmp[1], &all_back);
  const int have = (int)min((long long)count + all_back, (long long)a.free_capacity);

  // Needs of the requests whose tokens fit their table row and the T rows.
  auto need_of = [&](int c, int n, long long row_end) -> long long {
    if (n < 0 || n > most - c || row_end > a.T) return -1;
    return blocks(c + n) - blocks(c);
  };
  long long need = 0, at = row0;
  for (int b = b0; b < b1; ++b) {
    const int n = fresh(b);
    at += max(n, 0);
    need += max(need_of(cached(b), n, at), 0ll);
  }
  const long long need0 = block_exclusive_scan<kPlanThreads / 64>(need, tmp[2], &all_need);

  long long upto = need0, taken = 0, given = back0;
  at = row0;
  for (int b = b0; b < b1; ++b) {
    const int n = fresh(b);
    const int c = cached(b);
    s_row[b] = clamp_int(at);
    s_need[b] = clamp_int(upto);
    s_back[b] = clamp_int(given);
    if (blockIdx.x == 0) a.cu_new[b] = clamp_int(at);
    at += max(n, 0);
    if (n < 0) given += blocks(c);
    const long long mine = need_of(c, n, at);
    upto += max(mine, 0ll);
    const bool ok = mine == 0 || (mine > 0 && upto <= have);
    if (mine > 0 && ok) taken = upto;
    s_len[b] = ok ? c : -1;
    if (blockIdx.x == 0) a.seq_lens[b] = n < 0 ? 0 : ok ? c + n : c;
  }
  // Whole numbers up to free_capacity.
  taken = wave_reduce((int)taken, [](int x, int y) { return max(x, y); });
  if ((tid & 63) == 0) tmp[3][tid >> 6] = taken;
  __syncthreads();
  taken = max(max(tmp[3][0], tmp[3][1]), max(tmp[3][2], tmp[3][3]));
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_new[a.B] = clamp_int(all_rows);
    *a.free_count_out = have - (int)taken;
  }

  // Block given back j-th, and the i-th one handed out.
  auto returned = [&](int j) {
    const int b = last_at_most(s_back, a.B, j);
    return a.table[(size_t)b * a.max_blocks + (j - s_back[b])];
  };
  auto popped = [&](int i) {
    const int e = have - 1 - i;
    return e >= count ? returned(e - count) : a.free_blocks[e];
  };
  const int step = gridDim.x * kPlanThreads;
  const int g = blockIdx.x * kPlanThreads + tid;
  const int used_rows = (int)min(all_rows, (long long)a.T);
  for (int t = g; t < a.T; t += step) {
    long long slot = -1;
    int p = -1;
    if (t < used_rows) {
      const int b = last_at_most(s_row, a.B, t);
      const int c = s_len[b];
      if (c >= 0) {
        p = c + (t - s_row[b]);
        const int j = fast_div(p, by_block), old = blocks(c);
        const int page = j < old ? a.table[(size_t)b * a.max_blocks + j] : popped(s_need[b] + j - old);
        slot = (long long)page * bs + (p - j * bs);
      }
    }
    a.slots[t] = slot;
    a.positions[t] = p;
  }
  for (int i = g; i < (int)taken; i += step) {
    const int b = last_at_most(s_need, a.B, i);
    const int old = blocks(s_len[b]);
    a.table[(size_t)b * a.max_blocks + old + (i - s_need[b])] = popped(i);
  }
  for (int j = g; j < have - count; j += step) a.free_blocks[count + j] = returned(j);
}

hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream) {
  if (a.B < 0 || a.B > kMaxRequests) return hipErrorInvalidValue;
  // One thread a token; more threads for wide tables, whose blocks may all
  // come back in one call.
  const long long items = std::max<long long>(a.T, (long long)a.B * a.max_blocks / 16);
  const int grid = (int)std::min<long long>(std::max<long long>((items + 255) / 256, 1), 128);
  paged_plan_kernel<<<grid, kPlanThreads, (size_t)a.B * 16, stream>>>(
      a, make_fast_div(a.block_size));
  return hipGetLastError();
}

}  // namespace mova

// C ABI of the paged key-value cache's operators: argument checks, workspace
// sizes and launches.  Declarations and contracts: include/mova.h.
#include <math.h>

#include "../../include/mova.h"
#include "paged.h"

namespace {

using namespace mova;

constexpr int kMaxT = 1 << 24;
constexpr long long kMaxSlots = 1ll << 40;       // pools that are only written
constexpr long long kMaxReadSlots = 0x7fffffff;  // pools that are read: slots in 32 bits
constexpr long long kMaxLen = 1ll << 30;         // max_blocks * block_size

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

bool aligned(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

int check_table(int B, int max_blocks, int block_size) {
  if (B < 0 || max_blocks <= 0 || block_size <= 0) return MOVA_ERR_INVALID_ARG;
  if (B > kMaxRequests || (long long)max_blocks * block_size > kMaxLen) return MOVA_ERR_UNSUPPORTED;
  return MOVA_OK;
}

// Heads of the operators that read the cache.
int check_read_heads(int n_heads, int n_kv_heads, int head_dim) {
  if (n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0) return MOVA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MOVA_ERR_UNSUPPORTED;
  if (n_kv_heads > (1 << 14) / head_dim || n_heads % n_kv_heads != 0 ||
      n_heads > (1 << 17) / head_dim)
    return MOVA_ERR_UNSUPPORTED;
  return MOVA_OK;
}

int check_pool(int num_blocks, int block_size) {
  if (num_blocks < 0 || block_size <= 0) return MOVA_ERR_INVALID_ARG;
  return (long long)num_blocks * block_size > kMaxReadSlots ? MOVA_ERR_UNSUPPORTED : MOVA_OK;
}

int check_dtype(int cache_dtype, const float* k_scale, const float* v_scale) {
  if (cache_dtype != MOVA_CACHE_BF16 && cache_dtype != MOVA_CACHE_FP8) return MOVA_ERR_INVALID_ARG;
  // Scales belong to the 8-bit pools.
  if (cache_dtype == MOVA_CACHE_BF16 && (k_scale != nullptr || v_scale != nullptr))
    return MOVA_ERR_INVALID_ARG;
  return aligned(k_scale, 4) && aligned(v_scale, 4) ? MOVA_OK : MOVA_ERR_INVALID_ARG;
}

int check_select(int B, int n_heads, int n_kv_heads, int head_dim, int max_blocks, int block_size,
                 int keep) {
  int rc = check_table(B, max_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  rc = check_read_heads(n_heads, n_kv_heads, head_dim);
  if (rc != MOVA_OK) return rc;
  if (keep <= 0) return MOVA_ERR_INVALID_ARG;
  return keep > (1 << 20) ? MOVA_ERR_UNSUPPORTED : MOVA_OK;
}

int check_attention(int B, int n_heads, int n_kv_heads, int head_dim, int max_blocks,
                    int block_size, int keep) {
  int rc = check_table(B, max_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  rc = check_read_heads(n_heads, n_kv_heads, head_dim);
  if (rc != MOVA_OK) return rc;
  if (keep < 0) return MOVA_ERR_INVALID_ARG;
  return (long long)keep * block_size > kMaxLen ? MOVA_ERR_UNSUPPORTED : MOVA_OK;
}

int check_chunk(int T, int B, int n_heads, int n_kv_heads, int head_dim, int max_blocks,
                int block_size) {
  if (T < 0) return MOVA_ERR_INVALID_ARG;
  int rc = check_table(B, max_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  rc = check_read_heads(n_heads, n_kv_heads, head_dim);
  if (rc != MOVA_OK) return rc;
  if (T > kMaxT) return MOVA_ERR_UNSUPPORTED;
  // The line of work counts keys of row tiles in 53 bits.
  return (double)T * n_heads * ((double)max_blocks * block_size) > 0x1p52 ? MOVA_ERR_UNSUPPORTED
                                                                          : MOVA_OK;
}

// Pools whose blocks the upkeep counts.
int check_upkeep(int B, int max_blocks, int block_size, int num_blocks, int free_capacity) {
  const int rc = check_table(B, max_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  if (num_blocks < 0 || free_capacity < 0) return MOVA_ERR_INVALID_ARG;
  return num_blocks > kMaxUpkeepBlocks ? MOVA_ERR_UNSUPPORTED : MOVA_OK;
}

size_t free_bytes(int num_blocks) { return align256(4 * free_scratch_words(num_blocks)); }
size_t compact_bytes(int num_blocks) { return align256(4 * compact_scratch_words(num_blocks)); }

size_t select_bytes(int B, int n_kv_heads, int max_blocks) {
  return align256(8 * select_scratch_words(B, n_kv_heads, max_blocks));
}

int check_workspace(const void* workspace, size_t have, size_t need) {
  if (need == 0) return MOVA_OK;
  if (workspace == nullptr || have < need) return MOVA_ERR_WORKSPACE;
  return aligned(workspace, 256) ? MOVA_OK : MOVA_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int mova_paged_plan(const int32_t* cached_lens, const int32_t* new_lens, int B, int T,
                    int block_size, int max_blocks, int32_t* block_table, int32_t* free_blocks,
                    int free_capacity, const int32_t* free_count, int32_t* free_count_out,
                    int32_t* seq_lens, int32_t* cu_new, int64_t* slot_mapping, int32_t* positions,
                    hipStream_t stream) {
  int rc = check_table(B, max_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  if (T < 0 || free_capacity < 0) return MOVA_ERR_INVALID_ARG;
  if (T > kMaxT) return MOVA_ERR_UNSUPPORTED;
  if ((B > 0 && (cached_lens == nullptr || new_lens == nullptr || block_table == nullptr ||
                 seq_lens == nullptr)) ||
      free_count == nullptr || free_count_out == nullptr || cu_new == nullptr ||
      (free_capacity > 0 && free_blocks == nullptr) ||
      (T > 0 && (slot_mapping == nullptr || positions == nullptr)))
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_blocks, 4) || !aligned(free_count, 4) || !aligned(free_count_out, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_new, 4) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 4))
    return MOVA_ERR_INVALID_ARG;
  // Every workgroup reads these while one of them writes the others.
  if (free_count == free_count_out || (B > 0 && (cached_lens == seq_lens || new_lens == seq_lens)))
    return MOVA_ERR_INVALID_ARG;
  const PlanArgs a{cached_lens, new_lens, B, T, block_size, max_blocks, block_table, free_blocks,
                   free_capacity, free_count, free_count_out, seq_lens, cu_new, slot_mapping,
                   positions};
  return launch_paged_plan(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

int mova_kv_store_paged(const void* k, const void* v, int T, int n_kv_heads, int head_dim,
                        void* k_cache, void* v_cache, int cache_dtype, const float* k_scale,
                        const float* v_scale, int num_blocks, int block_size,
                        const int64_t* slot_mapping, void* k_bounds, hipStream_t stream) {
  if (T < 0 || n_kv_heads <= 0 || head_dim <= 0 || num_blocks < 0 || block_size <= 0)
    return MOVA_ERR_INVALID_ARG;
  if (T > kMaxT || head_dim % 16 != 0 || (long long)n_kv_heads * head_dim > (1 << 14) ||
      (long long)num_blocks * block_size > kMaxSlots)
    return MOVA_ERR_UNSUPPORTED;
  int rc = check_dtype(cache_dtype, k_scale, v_scale);
  if (rc != MOVA_OK) return rc;
  if (T == 0) return MOVA_OK;
  if ((k == nullptr && v == nullptr) || (k == nullptr) != (k_cache == nullptr) ||
      (v == nullptr) != (v_cache == nullptr) || (k_bounds != nullptr && k == nullptr) ||
      slot_mapping == nullptr)
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_bounds, 16) || !aligned(slot_mapping, 8))
    return MOVA_ERR_INVALID_ARG;
  const StoreArgs a{(const __bf16*)k, (const __bf16*)v, T, n_kv_heads, head_dim, k_cache, v_cache,
                    cache_dtype, k_scale, v_scale, (long long)num_blocks * block_size, block_size,
                    slot_mapping, (__bf16*)k_bounds};
  return launch_kv_store(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

size_t mova_block_select_workspace_bytes(int B, int n_heads, int n_kv_heads, int head_dim,
                                         int max_blocks, int block_size, int keep) {
  if (check_select(B, n_heads, n_kv_heads, head_dim, max_blocks, block_size, keep) != MOVA_OK)
    return (size_t)-1;
  return select_bytes(B, n_kv_heads, max_blocks);
}

int mova_block_select(const void* q, const void* k_bounds, int num_blocks, int block_size,
                      const int32_t* block_table, int max_blocks, const int32_t* seq_lens, int B,
                      int n_heads, int n_kv_heads, int head_dim, int keep, int keep_first,
                      int keep_last, int32_t* sel_blocks, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  int rc = check_select(B, n_heads, n_kv_heads, head_dim, max_blocks, block_size, keep);
  if (rc != MOVA_OK) return rc;
  rc = check_pool(num_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  if (keep_first < 0 || keep_last < 0 || keep_first > keep || keep_last > keep - keep_first)
    return MOVA_ERR_INVALID_ARG;
  if (B == 0) return MOVA_OK;
  if (q == nullptr || k_bounds == nullptr || block_table == nullptr || seq_lens == nullptr ||
      sel_blocks == nullptr)
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_bounds, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(sel_blocks, 4))
    return MOVA_ERR_INVALID_ARG;
  rc = check_workspace(workspace, workspace_bytes, select_bytes(B, n_kv_heads, max_blocks));
  if (rc != MOVA_OK) return rc;
  const SelectArgs a{(const __bf16*)q, (const __bf16*)k_bounds, num_blocks, block_size,
                     block_table, max_blocks, seq_lens, B, n_heads, n_kv_heads, head_dim, keep,
                     keep_first, keep_last, sel_blocks, (unsigned long long*)workspace};
  return launch_block_select(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

size_t mova_attention_workspace_bytes(int B, int n_heads, int n_kv_heads, int head_dim,
                                      int max_blocks, int block_size, int keep) {
  if (check_attention(B, n_heads, n_kv_heads, head_dim, max_blocks, block_size, keep) != MOVA_OK)
    return (size_t)-1;
  return align256(4 * attention_scratch_floats(B, n_heads, n_kv_heads, head_dim));
}

int mova_attention_paged(const void* q, const void* k_cache, const void* v_cache, int cache_dtype,
                         const float* k_scale, const float* v_scale, int num_blocks,
                         int block_size, const int32_t* block_table, int max_blocks,
                         const int32_t* seq_lens, const int32_t* sel_blocks, int keep, int B,
                         int n_heads, int n_kv_heads, int head_dim, float scale, int window,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  int rc = check_attention(B, n_heads, n_kv_heads, head_dim, max_blocks, block_size, keep);
  if (rc != MOVA_OK) return rc;
  rc = check_pool(num_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  rc = check_dtype(cache_dtype, k_scale, v_scale);
  if (rc != MOVA_OK) return rc;
  if (window < 0 || (keep == 0) != (sel_blocks == nullptr)) return MOVA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return MOVA_ERR_UNSUPPORTED;
  if (B == 0) return MOVA_OK;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_table == nullptr ||
      seq_lens == nullptr || out == nullptr)
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(sel_blocks, 4) ||
      !aligned(out, 16) || !aligned(lse, 4))
    return MOVA_ERR_INVALID_ARG;
  const size_t need = mova_attention_workspace_bytes(B, n_heads, n_kv_heads, head_dim, max_blocks,
                                                     block_size, keep);
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != MOVA_OK) return rc;
  const AttentionArgs a{(const __bf16*)q, k_cache, v_cache, cache_dtype, k_scale, v_scale,
                        num_blocks, block_size, block_table, max_blocks, seq_lens, sel_blocks,
                        keep, B, n_heads, n_kv_heads, head_dim, scale, window, (__bf16*)out, lse,
                        (float*)workspace};
  return launch_attention(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

size_t mova_attention_chunk_workspace_bytes(int T, int B, int n_heads, int n_kv_heads,
                                            int head_dim, int max_blocks, int block_size) {
  if (check_chunk(T, B, n_heads, n_kv_heads, head_dim, max_blocks, block_size) != MOVA_OK)
    return (size_t)-1;
  return align256(4 * chunk_scratch_floats(T, B, n_heads, n_kv_heads, head_dim,
                                           (long long)max_blocks * block_size));
}

int mova_attention_chunk_paged(const void* q, const void* k_cache, const void* v_cache,
                               int cache_dtype, const float* k_scale, const float* v_scale,
                               int num_blocks, int block_size, const int32_t* block_table,
                               int max_blocks, const int32_t* cached_lens, const int32_t* seq_lens,
                               const int32_t* cu_new, int T, int B, int n_heads, int n_kv_heads,
                               int head_dim, float scale, int window, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_chunk(T, B, n_heads, n_kv_heads, head_dim, max_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  rc = check_pool(num_blocks, block_size);
  if (rc != MOVA_OK) return rc;
  rc = check_dtype(cache_dtype, k_scale, v_scale);
  if (rc != MOVA_OK) return rc;
  if (window < 0) return MOVA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return MOVA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return MOVA_OK;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_table == nullptr ||
      cached_lens == nullptr || seq_lens == nullptr || cu_new == nullptr || out == nullptr)
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(cached_lens, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_new, 4) || !aligned(out, 16) || !aligned(lse, 4))
    return MOVA_ERR_INVALID_ARG;
  // Several workgroups read a row of q, at different times.
  if (out == q) return MOVA_ERR_INVALID_ARG;
  const size_t need = mova_attention_chunk_workspace_bytes(T, B, n_heads, n_kv_heads, head_dim,
                                                           max_blocks, block_size);
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != MOVA_OK) return rc;
  const ChunkArgs a{(const __bf16*)q, k_cache, v_cache, cache_dtype, k_scale, v_scale, num_blocks,
                    block_size, block_table, max_blocks, cached_lens, seq_lens, cu_new, T, B,
                    n_heads, n_kv_heads, head_dim, scale, window, (__bf16*)out, lse,
                    (float*)workspace};
  return launch_chunk_attention(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

int mova_paged_copy(const int32_t* copy_src, const int32_t* copy_dst, int n,
                    const int32_t* copy_count, void* k_cache, void* v_cache, void* k_bounds,
                    int cache_dtype, int num_blocks, int block_size, int n_kv_heads, int head_dim,
                    hipStream_t stream) {
  if (n < 0 || num_blocks < 0 || block_size <= 0 || n_kv_heads <= 0 || head_dim <= 0)
    return MOVA_ERR_INVALID_ARG;
  // A block's bytes in 16-byte pieces stay within 32 bits.
  if (head_dim % 16 != 0 || (long long)n_kv_heads * head_dim > (1 << 14) ||
      block_size > (1 << 18) || (long long)num_blocks * block_size > kMaxSlots)
    return MOVA_ERR_UNSUPPORTED;
  const int rc = check_dtype(cache_dtype, nullptr, nullptr);
  if (rc != MOVA_OK) return rc;
  if (n == 0) return MOVA_OK;
  if (copy_src == nullptr || copy_dst == nullptr ||
      (k_cache == nullptr && v_cache == nullptr && k_bounds == nullptr))
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(copy_count, 4) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_bounds, 16))
    return MOVA_ERR_INVALID_ARG;
  const int width = n_kv_heads * head_dim;
  const int rows = block_size * (width / (cache_dtype == MOVA_CACHE_FP8 ? 16 : 8));
  const CopyArgs a{copy_src, copy_dst, copy_count, n,
                   {(u32x4*)k_cache, (u32x4*)v_cache, (u32x4*)k_bounds},
                   {k_cache == nullptr ? 0 : rows, v_cache == nullptr ? 0 : rows,
                    k_bounds == nullptr ? 0 : width / 4},
                   num_blocks};
  return launch_paged_copy(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

int mova_paged_fork(const int32_t* parents, const int32_t* children, const int32_t* fork_lens,
                    int n, const int32_t* cached_lens, int B, int block_size, int max_blocks,
                    int32_t* block_table, const int32_t* free_blocks, int free_capacity,
                    const int32_t* free_count, int32_t* free_count_out, int32_t* shares,
                    int num_blocks, int32_t* seq_lens, int32_t* copy_src, int32_t* copy_dst,
                    hipStream_t stream) {
  const int rc = check_upkeep(B, max_blocks, block_size, num_blocks, free_capacity);
  if (rc != MOVA_OK) return rc;
  if (n < 0) return MOVA_ERR_INVALID_ARG;
  if (n > kMaxRequests) return MOVA_ERR_UNSUPPORTED;
  if ((B > 0 && (cached_lens == nullptr || block_table == nullptr || seq_lens == nullptr)) ||
      (n > 0 && (parents == nullptr || children == nullptr || copy_src == nullptr ||
                 copy_dst == nullptr)) ||
      free_count == nullptr || free_count_out == nullptr ||
      (free_capacity > 0 && free_blocks == nullptr) || (num_blocks > 0 && shares == nullptr))
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(fork_lens, 4) ||
      !aligned(cached_lens, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
      !aligned(free_count, 4) || !aligned(free_count_out, 4) || !aligned(shares, 4) ||
      !aligned(seq_lens, 4) || !aligned(copy_src, 4) || !aligned(copy_dst, 4))
    return MOVA_ERR_INVALID_ARG;
  // Every workgroup reads these while one of them writes the others.
  if (free_count == free_count_out || (B > 0 && cached_lens == seq_lens) ||
      (n > 0 && (fork_lens == seq_lens || copy_src == copy_dst)))
    return MOVA_ERR_INVALID_ARG;
  const ForkArgs a{parents, children, fork_lens, n, cached_lens, B, block_size, max_blocks,
                   block_table, free_blocks, free_capacity, free_count, free_count_out, shares,
                   num_blocks, seq_lens, copy_src, copy_dst};
  return launch_paged_fork(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

size_t mova_paged_free_workspace_bytes(int num_blocks) {
  if (num_blocks < 0 || num_blocks > kMaxUpkeepBlocks) return (size_t)-1;
  return free_bytes(num_blocks);
}

int mova_paged_free(const int32_t* cached_lens, const int32_t* keep_lens, int B, int block_size,
                    int max_blocks, const int32_t* block_table, int32_t* free_blocks,
                    int free_capacity, const int32_t* free_count, int32_t* free_count_out,
                    int32_t* shares, int num_blocks, int32_t* seq_lens, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  int rc = check_upkeep(B, max_blocks, block_size, num_blocks, free_capacity);
  if (rc != MOVA_OK) return rc;
  if ((B > 0 && (cached_lens == nullptr || keep_lens == nullptr || block_table == nullptr ||
                 seq_lens == nullptr)) ||
      free_count == nullptr || free_count_out == nullptr ||
      (free_capacity > 0 && free_blocks == nullptr) || (num_blocks > 0 && shares == nullptr))
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(cached_lens, 4) || !aligned(keep_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_blocks, 4) || !aligned(free_count, 4) || !aligned(free_count_out, 4) ||
      !aligned(shares, 4) || !aligned(seq_lens, 4))
    return MOVA_ERR_INVALID_ARG;
  if (free_count == free_count_out ||
      (B > 0 && (cached_lens == seq_lens || keep_lens == seq_lens)))
    return MOVA_ERR_INVALID_ARG;
  rc = check_workspace(workspace, workspace_bytes, free_bytes(num_blocks));
  if (rc != MOVA_OK) return rc;
  const FreeArgs a{cached_lens, keep_lens, B, block_size, max_blocks, block_table, free_blocks,
                   free_capacity, free_count, free_count_out, shares, num_blocks, seq_lens,
                   (uint32_t*)workspace};
  return launch_paged_free(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

size_t mova_paged_compact_workspace_bytes(int num_blocks) {
  if (num_blocks < 0 || num_blocks > kMaxUpkeepBlocks) return (size_t)-1;
  return compact_bytes(num_blocks);
}

int mova_paged_compact(const int32_t* cached_lens, int B, int block_size, int max_blocks,
                       const int32_t* block_table, int32_t* block_table_out,
                       const int32_t* free_blocks, int32_t* free_blocks_out, int free_capacity,
                       const int32_t* free_count, int32_t* free_count_out, const int32_t* shares,
                       int32_t* shares_out, int num_blocks, int limit, int32_t* remap,
                       int32_t* move_src, int32_t* move_dst, int32_t* move_count, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  int rc = check_upkeep(B, max_blocks, block_size, num_blocks, free_capacity);
  if (rc != MOVA_OK) return rc;
  if (limit < 0) return MOVA_ERR_INVALID_ARG;
  if ((B > 0 &&
       (cached_lens == nullptr || block_table == nullptr || block_table_out == nullptr)) ||
      free_count == nullptr || free_count_out == nullptr || move_count == nullptr ||
      (free_capacity > 0 && (free_blocks == nullptr || free_blocks_out == nullptr)) ||
      (num_blocks > 0 && (shares == nullptr || shares_out == nullptr || remap == nullptr)) ||
      (num_blocks > 1 && (move_src == nullptr || move_dst == nullptr)))
    return MOVA_ERR_INVALID_ARG;
  if (!aligned(cached_lens, 4) || !aligned(block_table, 4) || !aligned(block_table_out, 4) ||
      !aligned(free_blocks, 4) || !aligned(free_blocks_out, 4) || !aligned(free_count, 4) ||
      !aligned(free_count_out, 4) || !aligned(shares, 4) || !aligned(shares_out, 4) ||
      !aligned(remap, 4) || !aligned(move_src, 4) || !aligned(move_dst, 4) ||
      !aligned(move_count, 4))
    return MOVA_ERR_INVALID_ARG;
  if (free_count == free_count_out) return MOVA_ERR_INVALID_ARG;
  rc = check_workspace(workspace, workspace_bytes, compact_bytes(num_blocks));
  if (rc != MOVA_OK) return rc;
  const CompactArgs a{cached_lens, B, block_size, max_blocks, block_table, block_table_out,
                      free_blocks, free_blocks_out, free_capacity, free_count, free_count_out,
                      shares, shares_out, num_blocks, limit, remap, move_src, move_dst, move_count,
                      (uint32_t*)workspace};
  return launch_paged_compact(a, stream) == hipSuccess ? MOVA_OK : MOVA_ERR_HIP;
}

}  // extern "C"

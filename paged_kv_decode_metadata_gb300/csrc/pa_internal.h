// Host-side interface between the C ABI (pa_api.cu) and the kernel translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pa.h"

namespace pa {

// Error-word bits of the cache operators, beside those of pa_common.cuh (include/pa.h).
constexpr unsigned int kErrKeptOutOfRange = 1u << 5;  // kept position, or the position it moves to
constexpr unsigned int kErrTreeParent = 1u << 6;      // parent of a drafted node, not an earlier node
constexpr unsigned int kErrTokenOutOfRange = 1u << 7;  // drafted token outside the vocabulary
constexpr unsigned int kErrNoProbability = 1u << 8;    // a target row without a positive probability
constexpr unsigned int kErrOutOfPages = 1u << 9;       // fewer free pages than were asked for
constexpr unsigned int kErrPageRefs = 1u << 10;        // a page shared or given back that nobody holds

struct MetadataParams {
  const void* req_pool_indices;  // int64 or int32 (idx64)
  const void* seq_lens;          // int64 or int32 (idx64)
  const int32_t* req_to_token;
  int64_t req_to_token_rows;
  int64_t req_to_token_stride;
  const int64_t* full_to_swa_mapping;  // nullptr: no sliding-window outputs
  int64_t mapping_len;
  const int64_t* out_cache_loc;
  int64_t num_out_tokens;  // valid prefix of out_cache_loc (already min'ed)
  const void* qlens;  // int64 or int32 (idx64)
  int32_t* cache_seqlens;
  int32_t* cu_seqlens_k;
  int32_t* cu_seqlens_q;
  int32_t* page_table;
  int64_t page_table_stride;
  int32_t* swa_page_table;
  int64_t swa_page_table_stride;
  int64_t* swa_out_cache_loc;
  int64_t swa_out_len;
  int32_t bs;
  int32_t seqlen_offset;
  int32_t max_seq_pages;
  int32_t page_size;
  int32_t q_mode;
  int32_t q_stride;
  bool idx64;  // index inputs are int64 (else int32)
  unsigned int* err;
  unsigned long long* ts;  // stage timestamps (instrumented builds only), else nullptr
};

struct SplitKParams {
  const void* q;  // bf16 [bs, Hq, 128]
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* cache_seqlens;
  int64_t num_pages;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t max_seq_pages;
  int32_t pages_per_split;
  int32_t num_splits;
  float q_scale;  // sm_scale * log2(e)
  // Several query tokens per request (tensor-core producer only): query rows of request
  // b are cu_seqlens_q[b] .. cu_seqlens_q[b+1], at most max_q_len of them; nullptr for
  // one query per request (row b).
  const int32_t* cu_seqlens_q;
  int32_t max_q_len;
  // Sliding window (tensor-core producer only): > 0 restricts query i of a request to
  // its `window` newest positions, starts the split partition at the page of the
  // request's first visible position, and skips pages whose table entry is -1.
  // pages_per_split is then counted over the window's pages.  0: whole context.
  int32_t window;
  int32_t bs;        // requests (the persistent form walks them itself)
  int32_t work_slot;  // persistent form: the work-claim counter this launch uses
  int32_t sm_count;  // SMs of the device (grids of at most this many blocks take the
                     // deep-pipeline configuration)
  int32_t hold_loads;  // instrumented build only: the TMA warp issues nothing (timeout test)
  int32_t no_persist;  // instrumented build only: one block per item (A/B test)
  float* m_out;
  float* l_out;
  float* acc_out;
  unsigned int* err;
  unsigned long long* ts;  // stage timestamps (instrumented builds only), else nullptr
};

struct ReduceParams {
  const float* m;
  const float* l;
  const float* acc;
  int64_t num_rows;  // bs * Hq
  int32_t num_splits;
  void* out;   // bf16 [num_rows, 128]
  float* lse;  // [num_rows] or nullptr
  unsigned long long* ts;  // stage timestamps (instrumented builds only), else nullptr
};

struct RopeParams {
  const void *q, *k, *v;  // bf16 rows, head h of token t at x + t * stride + h * 128
  int64_t q_stride, k_stride, v_stride;
  const int64_t* positions;
  const int64_t* slots;
  const double* inv_freq;
  int32_t rotary_dim;
  float amplitude;
  int32_t num_tokens, num_q_heads, num_kv_heads;
  void* q_out;
  int64_t q_out_stride;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;  // int8 pools only
  float* weights;            // nullptr, or accumulated weights: 0 for the rows written
  int32_t page_size;
  int64_t num_pages;
  unsigned int* err;
};

struct RopeBlocksParams {
  const void *q, *k, *v;  // bf16 rows, head h of token t at x + t * stride + h * 128
  int64_t q_stride, k_stride, v_stride;
  const int64_t* positions;
  const double* inv_freq;
  int32_t rotary_dim;
  float amplitude;
  const int32_t* cu_seqlens_q;
  const int32_t* cache_seqlens;
  const int32_t* page_table;
  int64_t page_table_stride;
  int32_t max_seq_pages;
  int32_t bs, total_q, max_q_len;
  int32_t num_q_heads, num_kv_heads;
  void* q_out;
  int64_t q_out_stride;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;        // [num_pages, Hkv, page_size >> block_shift]
  int32_t page_shift, block_shift;  // log2 of the page size, of a scale's tokens
  int64_t num_pages;
  unsigned int* err;
};

struct TreeMaskParams {
  const int32_t* parents;
  const int32_t* cu_seqlens_q;
  int32_t bs, total_q, max_q_len;
  int64_t* tree_mask;
  int32_t mask_words;
  unsigned int* err;
};

// Chunks (of 128 tokens) that a piece of a tree's context has at most, where num_splits allows
// it: the tensor cores truncate each 4 tokens' sum as they add it to the accumulator, so n near-
// equal weights of one sign lose about n 2^-28, n 2^-25 at most.  (Whole contexts of 4M tokens
// read 1.1 % low, of 16M 3.9 %; in pieces of this length, nothing that bf16 shows.)
constexpr int32_t kTreePieceChunks = 2048;

struct TreeParams {
  const void* q;  // bf16 [total_q, Hq, 128]
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* cache_seqlens;
  const int32_t* cu_seqlens_q;
  const uint32_t* tree_mask;  // 2 * mask_words 32-bit words a row
  int32_t mask_words;
  int32_t bs, total_q, max_q_len;
  int32_t num_q_heads, num_kv_heads;
  int64_t num_pages;
  int32_t max_seq_pages;
  int32_t num_splits;  // most pieces of a row's context (partial slots per row)
  int32_t blocks;
  int32_t group_shift;  // log2 of the query heads per kv head
  float q_scale;  // sm_scale * log2(e)
  int32_t hold_loads;  // instrumented build only: three tiles, then no more (timeout test)
  // partials of several splits, or (one split) the output itself
  float *m_out, *l_out, *acc_out;
  void* out;
  float* lse;
  unsigned int* err;
};

struct BlockParams {
  const void* q;  // bf16 [total_q, Hq, 128]
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;  // [num_pages, Hkv, page_size >> block_shift]
  int32_t page_shift, block_shift;  // log2 of the page size, of a scale's tokens
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* cache_seqlens;
  const int32_t* cu_seqlens_q;  // nullptr: one query per request
  int32_t bs, total_q, max_q_len;
  int32_t num_q_heads, num_kv_heads, group;
  int64_t num_pages;
  int32_t max_seq_pages;
  int32_t tile_queries;  // queries of a tile: its columns are those times the group
  int32_t num_splits;  // most pieces of a row's context (partial slots per row)
  int32_t sm_count;
  int64_t line;        // chunks of the batch at most
  float q_scale;       // sm_scale * log2(e)
  int32_t hold_loads;  // instrumented build only: three tiles, then no more (timeout test)
  // partials of several splits, or (one split) the output itself
  float *m_out, *l_out, *acc_out;
  void* out;
  float* lse;
  unsigned int* err;
};

struct VerifyParams {
  const float* target_probs;
  int64_t target_stride;
  const float* draft_probs;  // nullptr: drafted tokens were proposed for certain
  int64_t draft_stride;
  int32_t vocab;
  const int64_t* tokens;
  const int32_t* parents;  // nullptr: chains
  const int32_t* cu_seqlens_q;
  const int32_t* cache_seqlens;  // nullptr: kept nodes are counted from 0
  const float *uniforms, *final_uniforms;
  int32_t bs, total_q, max_q_len;
  int32_t* kept;
  int64_t kept_stride;
  int32_t* counts;
  int32_t* begin;  // nullptr: not written
  int64_t* next_tokens;
  unsigned int* err;
};

// The page operators; each uses what it needs.
struct PagesParams {
  int32_t* req_to_token;
  int64_t num_rows, row_stride;
  int32_t* page_refs;
  int64_t num_pages, num_dst_pages;
  int32_t page_size, max_seq_pages;
  const int64_t *rows, *children;  // table rows (forks: the parents', the children's)
  const int32_t *lens, *new_lens;  // (free: tokens held, tokens kept, or nullptr)
  int32_t count;
  int32_t* granted;
  int32_t *src_pages, *dst_pages;  // copies; extend: first of a request's pages in `list`, how many
  int32_t* list;                   // free pages
  int32_t* page_map;
  int32_t* num_live;
  int32_t* num_moves;  // compaction: copies, counted on the device; else nullptr: `count`
  unsigned int* err;
};

// Up to kMax pools of a copy: the large ones (in tasks of part of a page) first.
struct PagesPools {
  static constexpr int kMax = 128;
  struct Pool {
    const void* src;
    void* dst;
    int64_t bytes;  // of a page
  };
  Pool pool[kMax];
  int32_t first_task[kMax + 1];
  int32_t num, large, tasks;
};

struct WeightsParams {
  const void* q;
  const float* lse;
  const void* k_cache;
  const float* k_scale;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* cache_seqlens;
  float* weights;
  int32_t bs, num_q_heads, num_kv_heads;
  int64_t num_pages;
  int32_t max_seq_pages;
  float q_scale;  // sm_scale * log2(e)
  unsigned int* err;
};

struct SelectParams {
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* cache_seqlens;
  int32_t max_seq_pages;
  const float* weights;
  int32_t budget, num_first, num_recent;
  int32_t* kept;
  int32_t* new_seqlens;
  int32_t bs, num_kv_heads, page_size;
  int64_t num_pages;
  unsigned int* err;
};

struct CompactParams {
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* cache_seqlens;
  int32_t max_seq_pages;
  const int32_t* kept;
  int32_t kept_heads;
  int64_t kept_stride;
  const int32_t* counts;
  const int32_t* begin;  // nullptr: 0
  int32_t max_kept;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale, *weights;  // nullptr where absent
  const int32_t* dst_page_table;
  int64_t dst_page_table_stride;
  int32_t dst_max_pages;
  int32_t* new_seqlens;  // nullptr: not written
  int32_t bs, num_kv_heads, page_size;
  int64_t num_pages;
  unsigned int* err;
};

// Step of the last failed launch on this host thread (for pa_last_error_string).
inline thread_local const char* g_fail_site = "launch";
inline cudaError_t fail_at(cudaError_t e, const char* site) {
  if (e != cudaSuccess) g_fail_site = site;
  return e;
}

// PA_OK for cudaSuccess; otherwise records `where`, the failed step and the CUDA error
// for pa_last_error_string on this host thread and returns PA_ERR_CUDA.
pa_status from_cuda(cudaError_t e, const char* where);

// Device address of the current device's error word (looked up once per device).
cudaError_t error_word(unsigned int** out);
int sm_count_of_current_device();
int32_t test_hold_loads();  // what pa_set_test_hold_loads was given (instrumented build; else 0)

// Argument checks shared by the entry points: the metadata stage's, and those of every
// attention over the pools (bs == 0 passes).
pa_status check_metadata(const void* req_pool_indices, const void* seq_lens,
                         const int32_t* req_to_token, int64_t req_to_token_rows,
                         int64_t req_to_token_stride, const int64_t* mapping, int64_t mapping_len,
                         int32_t* cache_seqlens, int32_t* cu_seqlens_k, int32_t* page_table,
                         int64_t page_table_stride, int32_t* swa_page_table,
                         int64_t swa_page_table_stride, int32_t bs, int32_t max_seq_pages,
                         int32_t page_size);
pa_status check_attention(const void* q, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, int32_t kv_dtype,
                          const int32_t* page_table, int64_t page_table_stride,
                          const int32_t* cache_seqlens, int32_t bs, int32_t num_q_heads,
                          int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                          int64_t num_pages, int32_t max_seq_pages, int32_t num_splits);

cudaError_t launch_metadata(const MetadataParams& p, cudaStream_t stream, bool use_pdl);

// bs, grid and shapes are validated by the caller.
cudaError_t launch_splitk_bf16(const SplitKParams& p, int bs, int group, int page_size,
                               cudaStream_t stream, bool use_pdl);
cudaError_t launch_splitk_int8(const SplitKParams& p, int bs, int group, int page_size,
                               cudaStream_t stream, bool use_pdl);

cudaError_t launch_splitk_mma_bf16(const SplitKParams& p, int bs, int group, int page_size,
                                   cudaStream_t stream, bool use_pdl);
cudaError_t launch_splitk_mma_int8(const SplitKParams& p, int bs, int group, int page_size,
                                   cudaStream_t stream, bool use_pdl);
// Sliding-window variants (SplitKParams::window > 0).
cudaError_t launch_splitk_mma_window_bf16(const SplitKParams& p, int bs, int group,
                                          int page_size, cudaStream_t stream, bool use_pdl);
cudaError_t launch_splitk_mma_window_int8(const SplitKParams& p, int bs, int group,
                                          int page_size, cudaStream_t stream, bool use_pdl);

cudaError_t launch_reduce(const ReduceParams& p, cudaStream_t stream, bool use_pdl);

cudaError_t launch_rope(const RopeParams& p, bool int8, bool interleaved, cudaStream_t stream,
                        bool use_pdl);
cudaError_t launch_rope_blocks(const RopeBlocksParams& p, bool interleaved, cudaStream_t stream,
                               bool use_pdl);
// Combines the partials that the tree attention left in `m_out`, `l_out` and `acc_out`.
cudaError_t launch_tree_join(const TreeParams& p, cudaStream_t stream, bool use_pdl);
cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t stream, bool use_pdl);
cudaError_t launch_tree_mma_bf16(const TreeParams& p, int group, int page_size,
                                 cudaStream_t stream, bool use_pdl);
cudaError_t launch_tree_mma_int8(const TreeParams& p, int group, int page_size,
                                 cudaStream_t stream, bool use_pdl);
cudaError_t launch_pages_copy(const PagesParams& p, const pa_page_pool* src, const pa_page_pool* dst,
                              int32_t from, int32_t num, int64_t most, cudaStream_t stream, bool use_pdl);
cudaError_t launch_pages_fork(const PagesParams& p, const pa_page_pool* pools, int32_t num,
                              cudaStream_t stream, bool use_pdl);
cudaError_t launch_pages_extend(const PagesParams& p, cudaStream_t stream, bool use_pdl);
cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t stream, bool use_pdl);
cudaError_t launch_pages_compact(const PagesParams& p, const pa_page_pool* pools, int32_t num,
                                 cudaStream_t stream, bool use_pdl);
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream, bool use_pdl);
// columns: (query, head) pairs of a tile, 8, 16 or 32.
cudaError_t launch_block(const BlockParams& p, int columns, cudaStream_t stream, bool use_pdl);
// Combines the partials of launch_block (num_splits > 1).
cudaError_t launch_block_join(const BlockParams& p, cudaStream_t stream, bool use_pdl);
cudaError_t launch_weights(const WeightsParams& p, bool int8, int group, int page_size,
                           cudaStream_t stream, bool use_pdl);
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream, bool use_pdl);
// in_place: the destination pages are the source pages.
cudaError_t launch_compact(const CompactParams& p, bool int8, bool in_place, cudaStream_t stream,
                           bool use_pdl);

}  // namespace pa

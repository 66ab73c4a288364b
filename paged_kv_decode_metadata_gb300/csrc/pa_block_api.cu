// C ABI of the block-scaled cache: append, attention, the step around it, split counts.  Argument
// checks and launches; see include/pa.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace {

constexpr int64_t kMaxPositions = int64_t{1} << 29;  // of a request: what kernels form stays int32
constexpr int32_t kMaxColumns = 32;                  // (query, head) pairs of a tile

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int32_t log2_of(int32_t x) {
  int32_t s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Columns of a tile (8, 16 or 32) for this group and query length, and the queries they hold.
int32_t tile_columns(int32_t group, int32_t max_q_len) {
  const int64_t want = static_cast<int64_t>(group) * max_q_len;
  return want <= 8 ? 8 : want <= 16 ? 16 : kMaxColumns;
}
int32_t tile_queries(int32_t group, int32_t max_q_len) {
  const int32_t fit = tile_columns(group, max_q_len) / group;
  return fit < max_q_len ? fit : max_q_len;
}

// Chunks (128 tokens of a tile of a kv head) of a batch of full lengths.
int64_t line_chunks(int32_t bs, int32_t max_q_len, int32_t group, int32_t num_kv_heads,
                    int32_t page_size, int32_t max_seq_pages) {
  const int64_t units = static_cast<int64_t>(bs) * num_kv_heads * cdiv(max_q_len, tile_queries(group, max_q_len));
  const int64_t chunks = cdiv(static_cast<int64_t>(max_seq_pages) * page_size, 128) + 2;  // (and what a unit costs beside them)
  return units > INT64_MAX / chunks ? INT64_MAX : units * chunks;
}

pa_status check_block_pools(const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, int32_t kv_dtype, int32_t scale_block,
                            const int32_t* page_table, int64_t page_table_stride,
                            const int32_t* cache_seqlens, int32_t bs, int32_t num_kv_heads,
                            int32_t head_dim, int32_t page_size, int64_t num_pages,
                            int32_t max_seq_pages) {
  if (kv_dtype != PA_KV_E4M3) return PA_ERR_INVALID;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !page_table || !cache_seqlens)
    return PA_ERR_INVALID;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(page_table, 4) || !aligned(cache_seqlens, 4))
    return PA_ERR_INVALID;
  if (num_kv_heads < 1 || num_kv_heads > 65535 || bs > 65535) return PA_ERR_INVALID;
  if (num_pages < 1 || max_seq_pages < 1 || page_table_stride < max_seq_pages)
    return PA_ERR_INVALID;
  if (head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return PA_ERR_UNSUPPORTED;
  if (scale_block != 16 && scale_block != 32 && scale_block != 64 && scale_block != 128)
    return PA_ERR_UNSUPPORTED;
  if (scale_block > page_size) return PA_ERR_INVALID;
  if (static_cast<int64_t>(max_seq_pages) * page_size > kMaxPositions) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Everything that pa_block_attention checks; *splits is the split count it will use.
pa_status check_block(const void* q, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, int32_t kv_dtype,
                      int32_t scale_block, const int32_t* page_table, int64_t page_table_stride,
                      const int32_t* cache_seqlens, const int32_t* cu_seqlens_q, int32_t bs,
                      int32_t total_q, int32_t max_q_len, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                      int64_t num_pages, int32_t max_seq_pages, int32_t num_splits,
                      float sm_scale, const void* workspace, size_t workspace_bytes,
                      const void* out, const float* lse, int32_t* splits) {
  if (num_splits < 0 || num_splits > 4096 || max_q_len < 1) return PA_ERR_INVALID;
  if (!q || !aligned(q, 16) || !out || !aligned(out, 16) || !aligned(lse, 4) || !aligned(cu_seqlens_q, 4))
    return PA_ERR_INVALID;
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
    return PA_ERR_INVALID;
  if (cu_seqlens_q == nullptr && (total_q != bs || max_q_len != 1)) return PA_ERR_INVALID;
  const pa_status st =
      check_block_pools(k_cache, v_cache, k_scale, v_scale, kv_dtype, scale_block, page_table,
                        page_table_stride, cache_seqlens, bs, num_kv_heads, head_dim, page_size,
                        num_pages, max_seq_pages);
  if (st != PA_OK) return st;
  if (!std::isfinite(sm_scale * 1.4426950408889634f)) return PA_ERR_INVALID;
  if (num_q_heads / num_kv_heads > kMaxColumns || max_q_len > 65535) return PA_ERR_UNSUPPORTED;
  // keeps the batch's chunks within 30 bits
  if (line_chunks(bs, max_q_len, num_q_heads / num_kv_heads, num_kv_heads, page_size, max_seq_pages) >=
      (int64_t{1} << 30))
    return PA_ERR_UNSUPPORTED;
  *splits = num_splits > 0 ? num_splits
                           : pa_choose_block_splits(bs, max_q_len, num_q_heads, num_kv_heads,
                                                    page_size, max_seq_pages, 0);
  if (*splits > 1 &&
      (!workspace || !aligned(workspace, 16) ||
       workspace_bytes < pa_workspace_bytes(total_q, num_q_heads, head_dim, *splits)))
    return PA_ERR_INVALID;
  return PA_OK;
}

pa_status finish(cudaError_t e, const char* where) {
  if (e == cudaSuccess) e = pa::fail_at(cudaGetLastError(), "error state after launch");
  return pa::from_cuda(e, where);
}

}  // namespace

extern "C" {

int32_t pa_choose_block_splits(int32_t bs, int32_t max_q_len, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t page_size, int32_t max_seq_pages,
                               int32_t sm_count) {
  if (bs <= 0 || max_q_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || page_size <= 0 ||
      max_seq_pages <= 0 || num_q_heads / num_kv_heads < 1 || num_q_heads / num_kv_heads > kMaxColumns)
    return 1;
  if (sm_count <= 0) sm_count = pa::sm_count_of_current_device();
  if (sm_count <= 0) sm_count = 152;
  // The batch's chunks of 128 tokens are shared out equally over the resident blocks, so a unit (a
  // tile of a kv head) longer than a share is cut.  Shares of a batch of equal lengths, and room
  // for one of half the length on average (a ragged one) before shares have to grow.
  const int32_t group = num_q_heads / num_kv_heads;
  const int32_t columns = tile_columns(group, max_q_len);
  const int64_t units = static_cast<int64_t>(bs) * num_kv_heads * cdiv(max_q_len, tile_queries(group, max_q_len));
  const int64_t chunks = cdiv(static_cast<int64_t>(max_seq_pages) * page_size, 128);
  const int64_t blocks = static_cast<int64_t>(sm_count) * (columns <= 16 ? 2 : 1);
  int64_t share = units * chunks / blocks;
  if (share < 1) share = 1;
  int64_t want = cdiv(2 * chunks, share) + 1;
  if (want > chunks) want = chunks;  // a piece holds a chunk at least
  if (want > 4096) want = 4096;
  return static_cast<int32_t>(want);
}

size_t pa_block_workspace_bytes(int32_t bs, int32_t total_q, int32_t max_q_len,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                int32_t page_size, int32_t max_seq_pages) {
  const int32_t splits =
      pa_choose_block_splits(bs, max_q_len, num_q_heads, num_kv_heads, page_size, max_seq_pages, 0);
  return splits > 1 ? pa_workspace_bytes(total_q, num_q_heads, head_dim, splits) : 0;
}

pa_status pa_rope_append_blocks(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const int64_t* positions, const double* inv_freq, int32_t rotary_dim,
    int32_t interleaved, float amplitude, const int32_t* cu_seqlens_q, const int32_t* cache_seqlens,
    const int32_t* page_table, int64_t page_table_stride, int32_t max_seq_pages, int32_t bs,
    int32_t total_q, int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
    float* k_scale, float* v_scale, int32_t kv_dtype, int32_t scale_block, int32_t page_size,
    int64_t num_pages, void* stream, int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0 || total_q == 0) return PA_OK;
  pa_status st = check_block_pools(k_cache, v_cache, k_scale, v_scale, kv_dtype, scale_block,
                                   page_table, page_table_stride, cache_seqlens, bs, num_kv_heads,
                                   head_dim, page_size, num_pages, max_seq_pages);
  if (st != PA_OK) return st;
  if (!cu_seqlens_q || !aligned(cu_seqlens_q, 4) || max_q_len < 1) return PA_ERR_INVALID;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return PA_ERR_INVALID;
  if (num_q_heads < 0 || num_q_heads > (1 << 20)) return PA_ERR_INVALID;
  if (rotary_dim != 0 && (!positions || !inv_freq || !aligned(positions, 8) || !aligned(inv_freq, 8)))
    return PA_ERR_INVALID;
  const int64_t strides[4] = {q_stride, k_stride, v_stride, q_out_stride};
  for (int i = 0; i < 4; ++i) {
    const int64_t heads = i == 0 || i == 3 ? num_q_heads : num_kv_heads;
    if (heads > 0 && (strides[i] % 8 != 0 || strides[i] < heads * 128)) return PA_ERR_INVALID;
  }
  if (num_q_heads > 0) {
    if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return PA_ERR_INVALID;
    if (q_out == q && q_out_stride != q_stride) return PA_ERR_INVALID;
  }
  if (!std::isfinite(amplitude)) return PA_ERR_INVALID;
  if (rotary_dim < 0 || rotary_dim > 128 || rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  pa::RopeBlocksParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.rotary_dim = rotary_dim;
  p.amplitude = amplitude;
  p.cu_seqlens_q = cu_seqlens_q;
  p.cache_seqlens = cache_seqlens;
  p.page_table = page_table;
  p.page_table_stride = page_table_stride;
  p.max_seq_pages = max_seq_pages;
  p.bs = bs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.q_out = q_out;
  p.q_out_stride = q_out_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.page_shift = log2_of(page_size);
  p.block_shift = log2_of(scale_block);
  p.num_pages = num_pages;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_rope_blocks(p, interleaved != 0, static_cast<cudaStream_t>(stream), use_pdl != 0),
                "block append launch");
}

pa_status pa_block_attention(const void* q, const void* k_cache, const void* v_cache,
                             const float* k_scale, const float* v_scale, int32_t kv_dtype,
                             int32_t scale_block, const int32_t* page_table,
                             int64_t page_table_stride, const int32_t* cache_seqlens,
                             const int32_t* cu_seqlens_q, int32_t bs, int32_t total_q,
                             int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
                             int32_t head_dim, int32_t page_size, int64_t num_pages,
                             int32_t max_seq_pages, int32_t num_splits, float sm_scale,
                             void* workspace, size_t workspace_bytes, void* out, float* lse,
                             void* stream, int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0 || total_q == 0) return PA_OK;
  int32_t splits = 1;
  pa_status st = check_block(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, scale_block,
                             page_table, page_table_stride, cache_seqlens, cu_seqlens_q, bs,
                             total_q, max_q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                             num_pages, max_seq_pages, num_splits, sm_scale, workspace,
                             workspace_bytes, out, lse, &splits);
  if (st != PA_OK) return st;
  const size_t rows = static_cast<size_t>(total_q) * num_q_heads * splits;
  char* ws = static_cast<char*>(workspace);
  pa::BlockParams p = {};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.page_shift = log2_of(page_size);
  p.block_shift = log2_of(scale_block);
  p.page_table = page_table;
  p.page_table_stride = page_table_stride;
  p.cache_seqlens = cache_seqlens;
  p.cu_seqlens_q = cu_seqlens_q;
  p.bs = bs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  p.num_pages = num_pages;
  p.max_seq_pages = max_seq_pages;
  p.tile_queries = tile_queries(p.group, max_q_len);
  p.num_splits = splits;
  p.sm_count = pa::sm_count_of_current_device();
  if (p.sm_count < 1) p.sm_count = 1;
  p.line = line_chunks(bs, max_q_len, p.group, num_kv_heads, page_size, max_seq_pages);
  p.q_scale = sm_scale * 1.4426950408889634f;  // log2(e): the kernel works in base 2
  p.hold_loads = pa::test_hold_loads();
  if (splits > 1) {
    p.m_out = reinterpret_cast<float*>(ws);
    p.l_out = reinterpret_cast<float*>(ws + align256(rows * sizeof(float)));
    p.acc_out = reinterpret_cast<float*>(ws + 2 * align256(rows * sizeof(float)));
  }
  p.out = out;
  p.lse = lse;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = finish(pa::launch_block(p, tile_columns(p.group, max_q_len), s, use_pdl != 0),
              "block attention launch");
  if (st != PA_OK || splits == 1) return st;
  return finish(pa::launch_block_join(p, s, use_pdl != 0), "block attention join launch");
}

pa_status pa_decode_step_block(
    const int64_t* req_pool_indices, const int64_t* seq_lens, const int32_t* req_to_token,
    int64_t req_to_token_rows, int64_t req_to_token_stride, const int64_t* full_to_swa_mapping,
    int64_t full_to_swa_mapping_len, int32_t seqlen_offset, int32_t max_seq_pages,
    int32_t* cache_seqlens, int32_t* cu_seqlens_k, int32_t* page_table, int64_t page_table_stride,
    int32_t* swa_page_table, int64_t swa_page_table_stride, const int64_t* qlens, int32_t q_mode,
    int32_t q_stride, int32_t* cu_seqlens_q, const void* q, int32_t total_q, int32_t max_q_len,
    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    int32_t kv_dtype, int32_t scale_block, int32_t bs, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t page_size, int64_t num_pages, int32_t num_splits, float sm_scale,
    void* workspace, size_t workspace_bytes, void* out, float* lse, void* stream,
    int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0) return PA_OK;
  if (total_q > 0) {
    int32_t splits = 1;
    pa_status st = check_block(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, scale_block,
                               page_table, page_table_stride, cache_seqlens, cu_seqlens_q, bs,
                               total_q, max_q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                               num_pages, max_seq_pages, num_splits, sm_scale, workspace,
                               workspace_bytes, out, lse, &splits);
    if (st != PA_OK) return st;
  }
  pa_status st = pa_build_metadata_full(
      req_pool_indices, seq_lens, 64, req_to_token, req_to_token_rows, req_to_token_stride,
      full_to_swa_mapping, full_to_swa_mapping_len, nullptr, 0, qlens, cache_seqlens, cu_seqlens_k,
      cu_seqlens_q, page_table, page_table_stride, swa_page_table, swa_page_table_stride, nullptr,
      0, bs, seqlen_offset, max_seq_pages, page_size, q_mode, q_stride, stream, use_pdl);
  if (st != PA_OK || total_q == 0) return st;
  return pa_block_attention(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, scale_block,
                            page_table, page_table_stride, cache_seqlens, cu_seqlens_q, bs, total_q,
                            max_q_len, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                            max_seq_pages, num_splits, sm_scale, workspace, workspace_bytes, out,
                            lse, stream, use_pdl);
}

}  // extern "C"

// C ABI of the cache operators: rotary append, tree attention, accumulated weights,
// compaction and eviction.  Argument checks and launches; see include/pa.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace {

constexpr int32_t kMaxTreeNodes = 256;
constexpr int64_t kMaxPositions = int64_t{1} << 30;  // of a request: positions plus a block stay int32

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool page_size_ok(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Both scales with an int8 pool; with bf16 they are ignored.
pa_status check_pools(const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, int32_t kv_dtype, int32_t num_kv_heads,
                      int32_t head_dim, int32_t page_size, int64_t num_pages) {
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_INT8) return PA_ERR_INVALID;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return PA_ERR_INVALID;
  if (kv_dtype == PA_KV_INT8 &&
      (!k_scale || !v_scale || !aligned(k_scale, 16) || !aligned(v_scale, 16)))
    return PA_ERR_INVALID;
  if (num_kv_heads < 1 || num_kv_heads > 65535 || num_pages < 1) return PA_ERR_INVALID;
  if (head_dim != 128 || !page_size_ok(page_size)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

pa_status finish(cudaError_t e, const char* where) {
  if (e == cudaSuccess) e = pa::fail_at(cudaGetLastError(), "error state after launch");
  return pa::from_cuda(e, where);
}

}  // namespace

extern "C" {

pa_status pa_rope_frequencies(double* inv_freq, int32_t rotary_dim, double base, int32_t scaling,
                              double factor, int64_t original_length, double low, double high) {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (inv_freq == nullptr || rotary_dim < 2 || rotary_dim % 2 != 0) return PA_ERR_INVALID;
  if (!std::isfinite(base) || !(base > 1.0)) return PA_ERR_INVALID;
  if (scaling < PA_ROPE_PLAIN || scaling > PA_ROPE_WAVELENGTH) return PA_ERR_INVALID;
  if (scaling != PA_ROPE_PLAIN && (!std::isfinite(factor) || !(factor > 0.0))) return PA_ERR_INVALID;
  if (scaling == PA_ROPE_BASE && rotary_dim == 2) return PA_ERR_INVALID;
  const bool split = scaling == PA_ROPE_BY_PARTS || scaling == PA_ROPE_WAVELENGTH;
  if (split && (original_length < 1 || !std::isfinite(low) || !std::isfinite(high) || !(low > 0.0) ||
                !(high > low)))
    return PA_ERR_INVALID;
  const double d = rotary_dim, len = static_cast<double>(original_length);
  if (scaling == PA_ROPE_BASE) base *= std::pow(factor, d / (d - 2.0));
  double lo = 0.0, hi = 0.0;
  if (scaling == PA_ROPE_BY_PARTS) {
    auto pair = [&](double turns) { return d * std::log(len / (kTwoPi * turns)) / (2.0 * std::log(base)); };
    lo = std::fmax(0.0, std::floor(pair(high)));
    hi = std::fmin(d - 1.0, std::ceil(pair(low)));
  }
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / d);
    double x = f;
    if (scaling == PA_ROPE_LINEAR) {
      x = f / factor;
    } else if (scaling == PA_ROPE_BY_PARTS) {
      const double r = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
      x = f * (1.0 - r) + f / factor * r;
    } else if (scaling == PA_ROPE_WAVELENGTH) {
      const double t = len * f / kTwoPi;
      const double s = std::fmin(1.0, std::fmax(0.0, (t - low) / (high - low)));
      x = t > high ? f : t < low ? f / factor : (1.0 - s) * f / factor + s * f;
    }
    inv_freq[i] = x;
  }
  return PA_OK;
}

pa_status pa_rope_append_weights(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                 const void* v, int64_t v_stride, const int64_t* positions,
                                 const int64_t* slots, const double* inv_freq, int32_t rotary_dim,
                                 int32_t interleaved, float amplitude, int32_t num_tokens,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out,
                                 int64_t q_out_stride, void* k_cache, void* v_cache, float* k_scale,
                                 float* v_scale, float* weights, int32_t kv_dtype, int32_t page_size,
                                 int64_t num_pages, void* stream, int32_t use_pdl) {
  if (num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  pa_status st = check_pools(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_kv_heads, head_dim,
                             page_size, num_pages);
  if (st != PA_OK) return st;
  if (!q || !k || !v || !positions || !slots || !inv_freq || !q_out) return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
    return PA_ERR_INVALID;
  if (!aligned(positions, 8) || !aligned(slots, 8) || !aligned(inv_freq, 8)) return PA_ERR_INVALID;
  if (num_q_heads < 1 || num_q_heads > (1 << 20)) return PA_ERR_INVALID;
  const int64_t strides[4] = {q_stride, k_stride, v_stride, q_out_stride};
  for (int i = 0; i < 4; ++i) {
    const int64_t heads = i == 0 || i == 3 ? num_q_heads : num_kv_heads;
    if (strides[i] % 8 != 0 || strides[i] < heads * 128) return PA_ERR_INVALID;
  }
  if (q_out == q && q_out_stride != q_stride) return PA_ERR_INVALID;
  if (!std::isfinite(amplitude)) return PA_ERR_INVALID;
  if (weights != nullptr && !aligned(weights, 4)) return PA_ERR_INVALID;
  if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  pa::RopeParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.rotary_dim = rotary_dim;
  p.amplitude = amplitude;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.q_out = q_out;
  p.q_out_stride = q_out_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.weights = weights;
  p.page_size = page_size;
  p.num_pages = num_pages;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_rope(p, kv_dtype == PA_KV_INT8, interleaved != 0,
                                static_cast<cudaStream_t>(stream), use_pdl != 0),
                "rotary append launch");
}

pa_status pa_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, const int64_t* positions,
                         const int64_t* slots, const double* inv_freq, int32_t rotary_dim,
                         int32_t interleaved, float amplitude, int32_t num_tokens,
                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out,
                         int64_t q_out_stride, void* k_cache, void* v_cache, float* k_scale,
                         float* v_scale, int32_t kv_dtype, int32_t page_size, int64_t num_pages,
                         void* stream, int32_t use_pdl) {
  return pa_rope_append_weights(q, q_stride, k, k_stride, v, v_stride, positions, slots, inv_freq,
                                rotary_dim, interleaved, amplitude, num_tokens, num_q_heads,
                                num_kv_heads, head_dim, q_out, q_out_stride, k_cache, v_cache,
                                k_scale, v_scale, nullptr, kv_dtype, page_size, num_pages, stream,
                                use_pdl);
}

pa_status pa_build_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, int32_t bs,
                             int32_t total_q, int32_t max_q_len, int64_t* tree_mask,
                             int32_t mask_words, void* stream, int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0 || total_q == 0) return PA_OK;
  if (!parents || !cu_seqlens_q || !tree_mask || !aligned(tree_mask, 8)) return PA_ERR_INVALID;
  if (max_q_len < 1 || mask_words < cdiv(max_q_len, 64)) return PA_ERR_INVALID;
  if (max_q_len > kMaxTreeNodes) return PA_ERR_UNSUPPORTED;
  pa::TreeMaskParams p = {};
  p.parents = parents;
  p.cu_seqlens_q = cu_seqlens_q;
  p.bs = bs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.tree_mask = tree_mask;
  p.mask_words = mask_words;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_tree_mask(p, static_cast<cudaStream_t>(stream), use_pdl != 0),
                "tree mask launch");
}

int32_t pa_choose_tree_splits(int32_t bs, int32_t max_q_len, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t page_size, int32_t max_seq_pages,
                              int32_t sm_count) {
  if (bs <= 0 || max_q_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || page_size <= 0 ||
      max_seq_pages <= 0)
    return 1;
  if (sm_count <= 0) sm_count = pa::sm_count_of_current_device();
  if (sm_count <= 0) sm_count = 152;
  // The batch's chunks of 128 tokens are shared out equally, so a unit (up to 256 rows of a
  // kv head) longer than a share is cut.  Shares of a batch of equal lengths, and room for
  // one of half the length on average (a ragged one) before shares have to grow.
  const int64_t group = num_q_heads / num_kv_heads > 0 ? num_q_heads / num_kv_heads : 1;
  const int64_t units = static_cast<int64_t>(bs) * num_kv_heads * cdiv(group * max_q_len, 256);
  const int64_t chunks = cdiv(static_cast<int64_t>(max_seq_pages) * page_size, 128);
  int64_t share = units * chunks / sm_count;
  if (share < 1) share = 1;
  int64_t want = cdiv(2 * chunks, share) + 1;
  // long contexts: pieces of half of the longest allowed, so that shares never grow past it
  if (chunks > pa::kTreePieceChunks) {
    const int64_t pieces = cdiv(2 * chunks, pa::kTreePieceChunks) + 1;
    if (want < pieces) want = pieces;
  }
  if (want > chunks) want = chunks;  // a piece holds a chunk at least
  if (want > 4096) want = 4096;
  return static_cast<int32_t>(want);
}

size_t pa_tree_workspace_bytes(int32_t bs, int32_t total_q, int32_t max_q_len, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               int32_t max_seq_pages) {
  const int32_t splits =
      pa_choose_tree_splits(bs, max_q_len, num_q_heads, num_kv_heads, page_size, max_seq_pages, 0);
  return splits > 1 ? pa_workspace_bytes(total_q, num_q_heads, head_dim, splits) : 0;
}

}  // extern "C"

namespace {

// Everything that pa_tree_attention checks; *splits is the split count it will use.
pa_status check_tree(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                     const float* v_scale, int32_t kv_dtype, const int32_t* page_table,
                     int64_t page_table_stride, const int32_t* cache_seqlens,
                     const int32_t* cu_seqlens_q, const int64_t* tree_mask, int32_t mask_words,
                     int32_t bs, int32_t total_q, int32_t max_q_len, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int64_t num_pages,
                     int32_t max_seq_pages, int32_t num_splits, float sm_scale,
                     const void* workspace, size_t workspace_bytes, const void* out,
                     int32_t* splits) {
  if (num_splits < 0 || max_q_len < 1 || mask_words < cdiv(max_q_len, 64)) return PA_ERR_INVALID;
  *splits = num_splits > 0 ? num_splits
                           : pa_choose_tree_splits(bs, max_q_len, num_q_heads, num_kv_heads,
                                                   page_size, max_seq_pages, 0);
  pa_status st = pa::check_attention(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, page_table,
                                     page_table_stride, cache_seqlens, bs, num_q_heads,
                                     num_kv_heads, head_dim, page_size, num_pages, max_seq_pages,
                                     *splits);
  if (st != PA_OK) return st;
  if (!cu_seqlens_q || !tree_mask || !aligned(tree_mask, 8)) return PA_ERR_INVALID;
  if (!out || !aligned(out, 16)) return PA_ERR_INVALID;
  if (!std::isfinite(sm_scale * 1.4426950408889634f) || !(sm_scale > 0.f)) return PA_ERR_INVALID;
  if (*splits > 1 &&
      (!workspace || !aligned(workspace, 16) ||
       workspace_bytes < pa_workspace_bytes(total_q, num_q_heads, head_dim, *splits)))
    return PA_ERR_INVALID;
  if (max_q_len > kMaxTreeNodes) return PA_ERR_UNSUPPORTED;
  // keeps every position the kernel forms within int32
  if (static_cast<int64_t>(max_seq_pages) * page_size > (int64_t{1} << 29)) return PA_ERR_UNSUPPORTED;
  // keeps a piece within 2^20 tokens, whose sums lose about as much as a bf16 rounding at most
  if (static_cast<int64_t>(max_seq_pages) * page_size > (int64_t{*splits > 1 ? *splits - 1 : 1} << 20))
    return PA_ERR_UNSUPPORTED;
  // keeps the batch's chunks (128 tokens of up to 256 rows of a kv head) within 31 bits
  const int64_t tiles = cdiv(static_cast<int64_t>(num_q_heads / num_kv_heads) * max_q_len, 256);
  const int64_t chunks = cdiv(static_cast<int64_t>(max_seq_pages) * page_size, 128);
  if (static_cast<int64_t>(bs) * num_kv_heads > INT32_MAX / 2 / (tiles * chunks)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale, int32_t kv_dtype,
                            const int32_t* page_table, int64_t page_table_stride,
                            const int32_t* cache_seqlens, const int32_t* cu_seqlens_q,
                            const int64_t* tree_mask, int32_t mask_words, int32_t bs,
                            int32_t total_q, int32_t max_q_len, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                            int64_t num_pages, int32_t max_seq_pages, int32_t num_splits,
                            float sm_scale, void* workspace, size_t workspace_bytes, void* out,
                            float* lse, void* stream, int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0 || total_q == 0) return PA_OK;
  int32_t splits = 1;
  pa_status st = check_tree(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, page_table,
                            page_table_stride, cache_seqlens, cu_seqlens_q, tree_mask, mask_words,
                            bs, total_q, max_q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                            num_pages, max_seq_pages, num_splits, sm_scale, workspace,
                            workspace_bytes, out, &splits);
  if (st != PA_OK) return st;
  const size_t rows = static_cast<size_t>(total_q) * num_q_heads * splits;
  char* ws = static_cast<char*>(workspace);
  pa::TreeParams p = {};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.page_table = page_table;
  p.page_table_stride = page_table_stride;
  p.cache_seqlens = cache_seqlens;
  p.cu_seqlens_q = cu_seqlens_q;
  p.tree_mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.mask_words = mask_words;
  p.bs = bs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_pages = num_pages;
  p.max_seq_pages = max_seq_pages;
  p.num_splits = splits;
  for (int g = num_q_heads / num_kv_heads; g > 1; g >>= 1) ++p.group_shift;
  const int64_t chunks = cdiv(static_cast<int64_t>(max_seq_pages) * page_size, 128);
  const int64_t most = static_cast<int64_t>(bs) * num_kv_heads *
                       cdiv(static_cast<int64_t>(num_q_heads / num_kv_heads) * max_q_len, 256) * chunks;
  int64_t sms = pa::sm_count_of_current_device();
  if (sms < 1) sms = 1;
  p.blocks = static_cast<int32_t>(most < sms ? most : sms);
  p.q_scale = sm_scale * 1.4426950408889634f;  // log2(e): the kernel works in base 2
  if (splits > 1) {
    p.m_out = reinterpret_cast<float*>(ws);
    p.l_out = reinterpret_cast<float*>(ws + align256(rows * sizeof(float)));
    p.acc_out = reinterpret_cast<float*>(ws + 2 * align256(rows * sizeof(float)));
  }
  p.out = out;
  p.lse = lse;
  p.hold_loads = pa::test_hold_loads();
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = finish((kv_dtype == PA_KV_INT8 ? pa::launch_tree_mma_int8 : pa::launch_tree_mma_bf16)(
                  p, num_q_heads / num_kv_heads, page_size, s, use_pdl != 0),
              "tree attention launch");
  if (st != PA_OK || splits == 1) return st;
  return finish(pa::launch_tree_join(p, s, use_pdl != 0), "tree join launch");
}

pa_status pa_decode_step_tree(
    const int64_t* req_pool_indices, const int64_t* seq_lens, const int32_t* req_to_token,
    int64_t req_to_token_rows, int64_t req_to_token_stride, const int64_t* full_to_swa_mapping,
    int64_t full_to_swa_mapping_len, int32_t seqlen_offset, int32_t max_seq_pages,
    int32_t* cache_seqlens, int32_t* cu_seqlens_k, int32_t* page_table, int64_t page_table_stride,
    int32_t* swa_page_table, int64_t swa_page_table_stride, const int64_t* qlens, int32_t q_mode,
    int32_t q_stride, int32_t* cu_seqlens_q, const int64_t* tree_mask, int32_t mask_words,
    const void* q, int32_t total_q, int32_t max_q_len, const void* k_cache, const void* v_cache,
    const float* k_scale, const float* v_scale, int32_t kv_dtype, int32_t bs, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int64_t num_pages,
    int32_t num_splits, float sm_scale, void* workspace, size_t workspace_bytes, void* out,
    float* lse, void* stream, int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0) return PA_OK;
  if (total_q > 0) {
    int32_t splits = 1;
    pa_status st = check_tree(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, page_table,
                              page_table_stride, cache_seqlens, cu_seqlens_q, tree_mask,
                              mask_words, bs, total_q, max_q_len, num_q_heads, num_kv_heads,
                              head_dim, page_size, num_pages, max_seq_pages, num_splits, sm_scale,
                              workspace, workspace_bytes, out, &splits);
    if (st != PA_OK) return st;
  }
  pa_status st = pa_build_metadata_full(
      req_pool_indices, seq_lens, 64, req_to_token, req_to_token_rows, req_to_token_stride,
      full_to_swa_mapping, full_to_swa_mapping_len, nullptr, 0, qlens, cache_seqlens, cu_seqlens_k,
      cu_seqlens_q, page_table, page_table_stride, swa_page_table, swa_page_table_stride, nullptr,
      0, bs, seqlen_offset, max_seq_pages, page_size, q_mode, q_stride, stream, use_pdl);
  if (st != PA_OK || total_q == 0) return st;
  return pa_tree_attention(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, page_table,
                           page_table_stride, cache_seqlens, cu_seqlens_q, tree_mask, mask_words,
                           bs, total_q, max_q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                           num_pages, max_seq_pages, num_splits, sm_scale, workspace,
                           workspace_bytes, out, lse, stream, use_pdl);
}

pa_status pa_accumulate_weights(const void* q, const float* lse, const void* k_cache,
                                const float* k_scale, int32_t kv_dtype, const int32_t* page_table,
                                int64_t page_table_stride, const int32_t* cache_seqlens,
                                float* weights, int32_t bs, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                                int64_t num_pages, int32_t max_seq_pages, float sm_scale,
                                void* stream, int32_t use_pdl) {
  // (K stands in for V, which this call does not have)
  pa_status st = pa::check_attention(q, k_cache, k_cache, k_scale, k_scale, kv_dtype, page_table,
                                     page_table_stride, cache_seqlens, bs, num_q_heads,
                                     num_kv_heads, head_dim, page_size, num_pages, max_seq_pages, 1);
  if (st != PA_OK || bs == 0) return st;
  if (!lse || !weights || !aligned(lse, 4) || !aligned(weights, 16)) return PA_ERR_INVALID;
  const float q_scale = sm_scale * 1.4426950408889634f;  // log2(e): the kernel works in base 2
  // (a sum that has become NaN stays it, and ranks above every other)
  if (!std::isfinite(q_scale)) return PA_ERR_INVALID;
  if (static_cast<int64_t>(max_seq_pages) * page_size > kMaxPositions) return PA_ERR_UNSUPPORTED;
  pa::WeightsParams p = {};
  p.q = q;
  p.lse = lse;
  p.k_cache = k_cache;
  p.k_scale = k_scale;
  p.page_table = page_table;
  p.page_table_stride = page_table_stride;
  p.cache_seqlens = cache_seqlens;
  p.weights = weights;
  p.bs = bs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_pages = num_pages;
  p.max_seq_pages = max_seq_pages;
  p.q_scale = q_scale;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_weights(p, kv_dtype == PA_KV_INT8, num_q_heads / num_kv_heads, page_size,
                                   static_cast<cudaStream_t>(stream), use_pdl != 0),
                "weights launch");
}

}  // extern "C"

namespace {

// Checks and the move's parameters common to compaction and eviction (bs >= 1).
pa_status compact_params(const int32_t* page_table, int64_t page_table_stride,
                         const int32_t* cache_seqlens, int32_t max_seq_pages, const int32_t* kept,
                         void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         int32_t kv_dtype, float* weights, const int32_t* dst_page_table,
                         int64_t dst_page_table_stride, int32_t dst_max_pages, int32_t bs,
                         int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                         int64_t num_pages, pa::CompactParams* p, bool* in_place) {
  pa_status st = check_pools(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_kv_heads, head_dim,
                             page_size, num_pages);
  if (st != PA_OK) return st;
  if (!page_table || !cache_seqlens || !dst_page_table) return PA_ERR_INVALID;
  if (bs > 65535 || max_seq_pages < 1 || page_table_stride < max_seq_pages || dst_max_pages < 1 ||
      dst_page_table_stride < dst_max_pages)
    return PA_ERR_INVALID;
  if (static_cast<int64_t>(max_seq_pages) * page_size > INT32_MAX ||
      static_cast<int64_t>(dst_max_pages) * page_size > INT32_MAX)
    return PA_ERR_INVALID;
  if (static_cast<int64_t>(max_seq_pages) * page_size > kMaxPositions) return PA_ERR_UNSUPPORTED;
  if (weights != nullptr && !aligned(weights, 4)) return PA_ERR_INVALID;
  *in_place = dst_page_table == page_table;
  if (*in_place && dst_page_table_stride != page_table_stride) return PA_ERR_INVALID;
  p->page_table = page_table;
  p->page_table_stride = page_table_stride;
  p->cache_seqlens = cache_seqlens;
  p->max_seq_pages = max_seq_pages;
  p->kept = kept;
  p->k_cache = k_cache;
  p->v_cache = v_cache;
  p->k_scale = kv_dtype == PA_KV_INT8 ? k_scale : nullptr;
  p->v_scale = kv_dtype == PA_KV_INT8 ? v_scale : nullptr;
  p->weights = weights;
  p->dst_page_table = dst_page_table;
  p->dst_page_table_stride = dst_page_table_stride;
  p->dst_max_pages = dst_max_pages;
  p->bs = bs;
  p->num_kv_heads = num_kv_heads;
  p->page_size = page_size;
  p->num_pages = num_pages;
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_compact_cache(const int32_t* page_table, int64_t page_table_stride,
                           const int32_t* cache_seqlens, int32_t max_seq_pages,
                           const int32_t* kept, int32_t kept_heads, int64_t kept_stride,
                           const int32_t* counts, const int32_t* begin, int32_t max_kept,
                           void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                           int32_t kv_dtype, float* weights, const int32_t* dst_page_table,
                           int64_t dst_page_table_stride, int32_t dst_max_pages,
                           int32_t* new_seqlens, int32_t bs, int32_t num_kv_heads,
                           int32_t head_dim, int32_t page_size, int64_t num_pages, void* stream,
                           int32_t use_pdl) {
  if (bs < 0) return PA_ERR_INVALID;
  if (bs == 0) return PA_OK;
  pa::CompactParams p = {};
  bool in_place = false;
  pa_status st = compact_params(page_table, page_table_stride, cache_seqlens, max_seq_pages, kept,
                                k_cache, v_cache, k_scale, v_scale, kv_dtype, weights,
                                dst_page_table, dst_page_table_stride, dst_max_pages, bs,
                                num_kv_heads, head_dim, page_size, num_pages, &p, &in_place);
  if (st != PA_OK) return st;
  if (!counts || max_kept < 0 || kept_stride < max_kept || (!kept && max_kept > 0))
    return PA_ERR_INVALID;
  if (kept_heads != 1 && kept_heads != num_kv_heads) return PA_ERR_INVALID;
  if (max_kept > kMaxPositions) return PA_ERR_UNSUPPORTED;
  // the blocks read these while one of them writes new_seqlens
  if (new_seqlens != nullptr && (new_seqlens == cache_seqlens || new_seqlens == counts || new_seqlens == begin))
    return PA_ERR_INVALID;
  p.kept_heads = kept_heads;
  p.kept_stride = kept_stride;
  p.counts = counts;
  p.begin = begin;
  p.max_kept = max_kept;
  p.new_seqlens = new_seqlens;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_compact(p, kv_dtype == PA_KV_INT8, in_place,
                                   static_cast<cudaStream_t>(stream), use_pdl != 0),
                "compaction launch");
}

pa_status pa_evict(const int32_t* page_table, int64_t page_table_stride,
                   const int32_t* cache_seqlens, int32_t max_seq_pages, float* weights,
                   void* k_cache, void* v_cache, float* k_scale, float* v_scale, int32_t kv_dtype,
                   int32_t budget, int32_t num_first, int32_t num_recent,
                   const int32_t* dst_page_table, int64_t dst_page_table_stride,
                   int32_t dst_max_pages, int32_t* kept, int32_t* new_seqlens, int32_t bs,
                   int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int64_t num_pages,
                   void* stream, int32_t use_pdl) {
  if (bs < 0) return PA_ERR_INVALID;
  if (bs == 0) return PA_OK;
  pa::CompactParams p = {};
  bool in_place = false;
  pa_status st = compact_params(page_table, page_table_stride, cache_seqlens, max_seq_pages, kept,
                                k_cache, v_cache, k_scale, v_scale, kv_dtype, weights,
                                dst_page_table, dst_page_table_stride, dst_max_pages, bs,
                                num_kv_heads, head_dim, page_size, num_pages, &p, &in_place);
  if (st != PA_OK) return st;
  if (!kept || !weights || !aligned(weights, 16) || !new_seqlens || new_seqlens == cache_seqlens)
    return PA_ERR_INVALID;
  if (budget < 1 || num_first < 0 || num_recent < 0 ||
      static_cast<int64_t>(num_first) + num_recent > budget)
    return PA_ERR_INVALID;
  const int64_t longest = static_cast<int64_t>(max_seq_pages) * page_size;
  if (static_cast<int64_t>(dst_max_pages) * page_size < (budget < longest ? budget : longest))
    return PA_ERR_INVALID;
  pa::SelectParams s = {};
  s.page_table = page_table;
  s.page_table_stride = page_table_stride;
  s.cache_seqlens = cache_seqlens;
  s.max_seq_pages = max_seq_pages;
  s.weights = weights;
  s.budget = budget;
  s.num_first = num_first;
  s.num_recent = num_recent;
  s.kept = kept;
  s.new_seqlens = new_seqlens;
  s.bs = bs;
  s.num_kv_heads = num_kv_heads;
  s.page_size = page_size;
  s.num_pages = num_pages;
  cudaError_t e = pa::error_word(&s.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  p.kept_heads = num_kv_heads;
  p.kept_stride = budget;
  p.counts = new_seqlens;
  p.max_kept = static_cast<int32_t>(budget < longest ? budget : longest);
  p.err = s.err;
  const cudaStream_t c = static_cast<cudaStream_t>(stream);
  st = finish(pa::launch_select(s, c, use_pdl != 0), "selection launch");
  if (st != PA_OK) return st;
  return finish(pa::launch_compact(p, kv_dtype == PA_KV_INT8, in_place, c, use_pdl != 0),
                "compaction launch");
}

}  // extern "C"

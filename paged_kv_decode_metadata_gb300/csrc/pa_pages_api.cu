// C ABI of the draft verification and of the page operators.  Argument checks and launches; see include/pa.h for the contract.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

pa_status finish(cudaError_t e, const char* where) {
  if (e == cudaSuccess) e = pa::fail_at(cudaGetLastError(), "error state after launch");
  return pa::from_cuda(e, where);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Pools of a copy; page counts are the caller's word.
pa_status check_pools(const pa_page_pool* pools, int32_t num_pools) {
  if (num_pools < 0 || (num_pools > 0 && !pools)) return PA_ERR_INVALID;
  for (int32_t i = 0; i < num_pools; ++i)
    if (!pools[i].base || !aligned(pools[i].base, 4) || pools[i].page_bytes < 4 || pools[i].page_bytes % 4 != 0)
      return PA_ERR_INVALID;
  return PA_OK;
}

// What the operators on the slot table have in common.
pa_status table_params(int32_t* req_to_token, int64_t num_rows, int64_t row_stride,
                       int32_t* page_refs, int64_t num_pages, int32_t page_size,
                       int32_t max_seq_pages, const int64_t* rows, const int32_t* lens,
                       int32_t count, pa::PagesParams* p) {
  if (!req_to_token || !page_refs || (count > 0 && (!rows || !lens))) return PA_ERR_INVALID;
  if (!aligned(req_to_token, 4) || !aligned(page_refs, 4) || !aligned(rows, 8) || !aligned(lens, 4))
    return PA_ERR_INVALID;
  if (num_rows < 1 || num_pages < 1 || page_size < 1 || max_seq_pages < 1) return PA_ERR_INVALID;
  if (static_cast<int64_t>(max_seq_pages - 1) * page_size >= row_stride) return PA_ERR_INVALID;
  if (num_pages > INT32_MAX / page_size) return PA_ERR_INVALID;  // slots are int32
  if (num_pages > (1 << 20) || count > 65535 ||
      static_cast<int64_t>(max_seq_pages) * page_size > (int64_t{1} << 29))
    return PA_ERR_UNSUPPORTED;
  p->req_to_token = req_to_token;
  p->num_rows = num_rows;
  p->row_stride = row_stride;
  p->page_refs = page_refs;
  p->num_pages = p->num_dst_pages = num_pages;
  p->page_size = page_size;
  p->max_seq_pages = max_seq_pages;
  p->rows = rows;
  p->lens = lens;
  p->count = count;
  return PA_OK;
}

// The workspace: a number, the copies' two lists, the free pages.
pa_status carve(void* workspace, size_t workspace_bytes, int64_t num_pages, int32_t count,
                pa::PagesParams* p, int32_t** number) {
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < pa_pages_workspace_bytes(num_pages, count))
    return PA_ERR_INVALID;
  char* at = static_cast<char*>(workspace);
  const size_t pairs = align256(sizeof(int32_t) * static_cast<size_t>(num_pages > count ? num_pages : count));
  *number = reinterpret_cast<int32_t*>(at);
  p->src_pages = reinterpret_cast<int32_t*>(at + 256);
  p->dst_pages = reinterpret_cast<int32_t*>(at + 256 + pairs);
  p->list = reinterpret_cast<int32_t*>(at + 256 + 2 * pairs);
  return PA_OK;
}

}  // namespace

extern "C" {

size_t pa_pages_workspace_bytes(int64_t num_pages, int32_t count) {
  if (num_pages < 0 || count < 0) return 0;
  const size_t pairs = align256(sizeof(int32_t) * static_cast<size_t>(num_pages > count ? num_pages : count));
  return 256 + 3 * pairs;
}

pa_status pa_pages_copy(const pa_page_pool* src_pools, const pa_page_pool* dst_pools,
                        int32_t num_pools, int64_t num_src_pages, int64_t num_dst_pages,
                        const int32_t* src_pages, const int32_t* dst_pages, int32_t count,
                        void* stream, int32_t use_pdl) {
  if (count < 0) return PA_ERR_INVALID;
  pa_status st = check_pools(src_pools, num_pools);
  if (st != PA_OK) return st;
  if (dst_pools == nullptr) dst_pools = src_pools;
  st = check_pools(dst_pools, num_pools);
  if (st != PA_OK) return st;
  for (int32_t i = 0; i < num_pools; ++i)
    if (src_pools[i].page_bytes != dst_pools[i].page_bytes) return PA_ERR_INVALID;
  if (count == 0 || num_pools == 0) return PA_OK;
  if (!src_pages || !dst_pages || !aligned(src_pages, 4) || !aligned(dst_pages, 4)) return PA_ERR_INVALID;
  if (num_src_pages < 1 || num_dst_pages < 1) return PA_ERR_INVALID;
  pa::PagesParams p = {};
  p.num_pages = num_src_pages;
  p.num_dst_pages = num_dst_pages;
  p.count = count;
  p.src_pages = const_cast<int32_t*>(src_pages);
  p.dst_pages = const_cast<int32_t*>(dst_pages);
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_pages_copy(p, src_pools, dst_pools, 0, num_pools, count,
                                      static_cast<cudaStream_t>(stream), use_pdl != 0),
                "page copy launch");
}

pa_status pa_pages_fork(int32_t* req_to_token, int64_t num_rows, int64_t row_stride,
                        int32_t* page_refs, int64_t num_pages, int32_t page_size,
                        int32_t max_seq_pages, const int64_t* parents, const int64_t* children,
                        const int32_t* lens, int32_t count, const pa_page_pool* pools,
                        int32_t num_pools, int32_t* child_lens, void* workspace,
                        size_t workspace_bytes, void* stream, int32_t use_pdl) {
  if (count < 0) return PA_ERR_INVALID;
  if (count == 0) return PA_OK;
  pa_status st = check_pools(pools, num_pools);
  if (st != PA_OK) return st;
  pa::PagesParams p = {};
  st = table_params(req_to_token, num_rows, row_stride, page_refs, num_pages, page_size,
                    max_seq_pages, parents, lens, count, &p);
  if (st != PA_OK) return st;
  int32_t* number = nullptr;
  if ((st = carve(workspace, workspace_bytes, num_pages, count, &p, &number)) != PA_OK) return st;
  if (!children || !aligned(children, 8) || !child_lens || !aligned(child_lens, 4) || child_lens == lens)
    return PA_ERR_INVALID;
  p.children = children;
  p.granted = child_lens;
  const cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_pages_fork(p, pools, num_pools, static_cast<cudaStream_t>(stream), use_pdl != 0),
                "page fork launch");
}

pa_status pa_pages_extend(int32_t* req_to_token, int64_t num_rows, int64_t row_stride,
                          int32_t* page_refs, int64_t num_pages, int32_t page_size,
                          int32_t max_seq_pages, const int64_t* rows, const int32_t* lens,
                          const int32_t* new_lens, int32_t count, int32_t* granted,
                          void* workspace, size_t workspace_bytes, void* stream, int32_t use_pdl) {
  if (count < 0) return PA_ERR_INVALID;
  if (count == 0) return PA_OK;
  pa::PagesParams p = {};
  pa_status st = table_params(req_to_token, num_rows, row_stride, page_refs, num_pages, page_size,
                              max_seq_pages, rows, lens, count, &p);
  if (st != PA_OK) return st;
  int32_t* number = nullptr;
  if ((st = carve(workspace, workspace_bytes, num_pages, count, &p, &number)) != PA_OK) return st;
  if (!new_lens || !granted || !aligned(new_lens, 4) || !aligned(granted, 4) || granted == lens ||
      granted == new_lens)
    return PA_ERR_INVALID;
  p.new_lens = new_lens;
  p.granted = granted;
  const cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_pages_extend(p, static_cast<cudaStream_t>(stream), use_pdl != 0),
                "page extend launch");
}

pa_status pa_pages_free(int32_t* req_to_token, int64_t num_rows, int64_t row_stride,
                        int32_t* page_refs, int64_t num_pages, int32_t page_size,
                        int32_t max_seq_pages, const int64_t* rows, const int32_t* lens,
                        const int32_t* keep_lens, int32_t count, void* stream, int32_t use_pdl) {
  if (count < 0) return PA_ERR_INVALID;
  if (count == 0) return PA_OK;
  pa::PagesParams p = {};
  const pa_status st = table_params(req_to_token, num_rows, row_stride, page_refs, num_pages,
                                    page_size, max_seq_pages, rows, lens, count, &p);
  if (st != PA_OK) return st;
  if (!aligned(keep_lens, 4)) return PA_ERR_INVALID;
  p.new_lens = keep_lens;
  const cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_pages_free(p, static_cast<cudaStream_t>(stream), use_pdl != 0),
                "page free launch");
}

pa_status pa_pages_compact(int32_t* req_to_token, int64_t num_rows, int64_t row_stride,
                           int32_t* page_refs, int64_t num_pages, int32_t page_size,
                           int32_t max_seq_pages, const int64_t* rows, const int32_t* lens,
                           int32_t count, const pa_page_pool* pools, int32_t num_pools,
                           int32_t* page_map, int32_t* num_live, void* workspace,
                           size_t workspace_bytes, void* stream, int32_t use_pdl) {
  if (count < 0) return PA_ERR_INVALID;
  pa_status st = check_pools(pools, num_pools);
  if (st != PA_OK) return st;
  pa::PagesParams p = {};
  st = table_params(req_to_token, num_rows, row_stride, page_refs, num_pages, page_size,
                    max_seq_pages, rows, lens, count, &p);
  if (st != PA_OK) return st;
  if ((st = carve(workspace, workspace_bytes, num_pages, count, &p, &p.num_moves)) != PA_OK) return st;
  if (!page_map || !num_live || !aligned(page_map, 4) || !aligned(num_live, 4)) return PA_ERR_INVALID;
  p.page_map = page_map;
  p.num_live = num_live;
  const cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_pages_compact(p, pools, num_pools, static_cast<cudaStream_t>(stream), use_pdl != 0),
                "page compaction launch");
}

pa_status pa_verify_drafts(const float* target_probs, int64_t target_stride,
                           const float* draft_probs, int64_t draft_stride, int32_t vocab,
                           const int64_t* tokens, const int32_t* parents,
                           const int32_t* cu_seqlens_q, const int32_t* cache_seqlens,
                           const float* uniforms, const float* final_uniforms, int32_t bs,
                           int32_t total_q, int32_t max_q_len, int32_t* kept, int64_t kept_stride,
                           int32_t* counts, int32_t* begin, int64_t* next_tokens, void* stream,
                           int32_t use_pdl) {
  if (bs < 0 || total_q < 0) return PA_ERR_INVALID;
  if (bs == 0) return PA_OK;
  // (no rows at all: the requests' results are still written)
  if (total_q > 0 && (!target_probs || !tokens || !uniforms)) return PA_ERR_INVALID;
  if (!cu_seqlens_q || !final_uniforms || !kept || !counts || !next_tokens) return PA_ERR_INVALID;
  if (!aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(tokens, 8) || !aligned(next_tokens, 8))
    return PA_ERR_INVALID;
  for (const void* x : {static_cast<const void*>(parents), static_cast<const void*>(cu_seqlens_q),
                        static_cast<const void*>(cache_seqlens), static_cast<const void*>(uniforms),
                        static_cast<const void*>(final_uniforms), static_cast<const void*>(kept),
                        static_cast<const void*>(counts), static_cast<const void*>(begin)})
    if (!aligned(x, 4)) return PA_ERR_INVALID;
  if (vocab < 1 || target_stride < vocab || (draft_probs && draft_stride < vocab)) return PA_ERR_INVALID;
  if (max_q_len < 1 || kept_stride < max_q_len || bs > 65535) return PA_ERR_INVALID;
  // the blocks read these while one of them writes the outputs
  if (cache_seqlens && (cache_seqlens == counts || cache_seqlens == begin)) return PA_ERR_INVALID;
  if (max_q_len > 256 || vocab > (1 << 20)) return PA_ERR_UNSUPPORTED;
  pa::VerifyParams p = {};
  p.target_probs = target_probs;
  p.target_stride = target_stride;
  p.draft_probs = draft_probs;
  p.draft_stride = draft_stride;
  p.vocab = vocab;
  p.tokens = tokens;
  p.parents = parents;
  p.cu_seqlens_q = cu_seqlens_q;
  p.cache_seqlens = cache_seqlens;
  p.uniforms = uniforms;
  p.final_uniforms = final_uniforms;
  p.bs = bs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.kept = kept;
  p.kept_stride = kept_stride;
  p.counts = counts;
  p.begin = begin;
  p.next_tokens = next_tokens;
  cudaError_t e = pa::error_word(&p.err);
  if (e != cudaSuccess) return pa::from_cuda(e, "error word lookup");
  return finish(pa::launch_verify(p, static_cast<cudaStream_t>(stream), use_pdl != 0), "verify launch");
}

}  // extern "C"

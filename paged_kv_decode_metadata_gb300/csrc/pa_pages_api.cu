// C ABI of the draft verification.  Argument checks and launches; see include/pa.h for the contract.
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

}  // namespace

extern "C" {

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
  if (!target_probs || !tokens || !cu_seqlens_q || !uniforms || !final_uniforms || !kept || !counts ||
      !next_tokens)
    return PA_ERR_INVALID;
  if (!aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(tokens, 8) || !aligned(next_tokens, 8))
    return PA_ERR_INVALID;
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

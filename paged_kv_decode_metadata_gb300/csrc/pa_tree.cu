// Ancestor masks of drafted trees, and the join of the partial results that the tree
// attention (pa_tree_mma.cuh) leaves of rows whose context was cut into pieces.
#include <math_constants.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// ---- ancestor masks ---------------------------------------------------------------------------

constexpr int kMaxNodes = 256;

// One block per request: its parents in shared memory, one thread per node walking up.
__global__ void __launch_bounds__(kMaxNodes) tree_mask_kernel(const TreeMaskParams p) {
  __shared__ int parent_s[kMaxNodes];
  const int b = blockIdx.x, i = threadIdx.x;
  grid_dependency_wait();
  const int begin = p.cu_seqlens_q[b];
  int q_len = p.cu_seqlens_q[b + 1] - begin;
  if (begin < 0 || q_len < 0 || q_len > p.max_q_len || begin > p.total_q - q_len) {
    if (i == 0) record_error(p.err, kErrSeqLenOutOfRange);
    q_len = 0;
  }
  if (i < q_len) {
    int up = p.parents[begin + i];
    if (up < -1 || up >= i) {
      record_error(p.err, kErrTreeParent);
      up = -1;
    }
    parent_s[i] = up;
  }
  __syncthreads();
  if (i >= q_len) return;
  uint64_t bits[kMaxNodes / 64] = {0, 0, 0, 0};
  for (int t = i; t >= 0; t = parent_s[t]) {  // (parents are earlier nodes: it ends)
#pragma unroll
    for (int w = 0; w < kMaxNodes / 64; ++w)
      if (t >> 6 == w) bits[w] |= 1ull << (t & 63);
  }
  int64_t* row = p.tree_mask + static_cast<int64_t>(begin + i) * p.mask_words;
  for (int w = 0; w < p.mask_words; ++w) {
    uint64_t v = 0;
#pragma unroll
    for (int u = 0; u < kMaxNodes / 64; ++u)
      if (u == w) v = bits[u];
    row[w] = static_cast<int64_t>(v);
  }
}

// ---- the join of a row's pieces ---------------------------------------------------------------

constexpr int kJoinWarps = 8;

// The list of a row's pieces is its l values up to the first negative one (or num_splits of
// them); a row whose first l is negative has its output already.  A warp looks at `per`
// rows at once and combines those that were cut, a lane owning 4 channels:
//   M = max m_s, out = sum acc_s e^(m_s - M) / sum l_s e^(m_s - M), lse = M + ln of that sum.
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const TreeParams p, int per) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 =
      (static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5)) * per;
  const int S = p.num_splits;
  grid_dependency_wait();
  const int64_t rows =
      static_cast<int64_t>(max(0, min(p.cu_seqlens_q[p.bs], p.total_q))) * p.num_q_heads;
  const bool cut = lane < per && row0 + lane < rows && !(p.l_out[(row0 + lane) * S] < 0.f);
  uint32_t todo = __ballot_sync(0xffffffffu, cut);
  while (todo != 0) {
    const int64_t row = row0 + __ffs(todo) - 1;
    todo &= todo - 1;
    const float* m = p.m_out + row * S;
    const float* l = p.l_out + row * S;
    const float4* acc = reinterpret_cast<const float4*>(p.acc_out) + row * S * 32 + lane;
    float top = -CUDART_INF_F, total = 0.f;
    bool nan = false;  // a piece had a NaN score: its sum is NaN, its maximum may be -inf
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += 32) {
      const float ls = s0 + lane < S ? l[s0 + lane] : -1.f;
      const uint32_t ends = __ballot_sync(0xffffffffu, ls < 0.f);
      const int count = ends != 0 ? __ffs(ends) - 1 : 32;
      const float ms = lane < count ? m[s0 + lane] : -CUDART_INF_F;
      nan = nan || __any_sync(0xffffffffu, lane < count && ls != ls);
      const float new_top = fmaxf(top, warp_max(ms));
      if (new_top != -CUDART_INF_F) {
        const float keep = top == -CUDART_INF_F ? 0.f : expf(top - new_top);
        const float w = ms == -CUDART_INF_F ? 0.f : expf(ms - new_top);
        total = total * keep + warp_sum(lane < count ? w * ls : 0.f);
        o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
        for (int s = 0; s < count; s += 4) {
          float4 a[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) a[u] = acc[(s0 + min(s + u, count - 1)) * 32];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float ws = __shfl_sync(0xffffffffu, w, min(s + u, count - 1));
            if (s + u < count && ws != 0.f) {
              o.x = fmaf(ws, a[u].x, o.x);
              o.y = fmaf(ws, a[u].y, o.y);
              o.z = fmaf(ws, a[u].z, o.z);
              o.w = fmaf(ws, a[u].w, o.w);
            }
          }
        }
        top = new_top;
      }
      if (count < 32) break;
    }
    if (nan) total = CUDART_NAN_F;
    const float inv = top == -CUDART_INF_F && !nan ? 0.f : 1.f / total;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    static_cast<uint2*>(p.out)[row * 32 + lane] = make_uint2(
        *reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (p.lse != nullptr && lane == 0)
      p.lse[row] = top == -CUDART_INF_F && !nan ? top : top + logf(total);
  }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t stream, bool use_pdl) {
  return fail_at(launch_kernel(tree_mask_kernel, dim3(p.bs), dim3(kMaxNodes), 0, stream, use_pdl, p),
                 "cudaLaunchKernelEx");
}

cudaError_t launch_tree_join(const TreeParams& p, cudaStream_t stream, bool use_pdl) {
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.num_q_heads;
  // rows per warp: few while there are not two rows a warp slot of the device
  int per = 1;
  while (per < 32 && rows / per > 152 * 64) per *= 2;
  const int64_t warps = (rows + per - 1) / per;
  return fail_at(launch_kernel(tree_join_kernel, dim3(static_cast<unsigned>((warps + kJoinWarps - 1) / kJoinWarps)),
                               dim3(kJoinWarps * 32), 0, stream, use_pdl, p, per),
                 "cudaLaunchKernelEx (join)");
}

}  // namespace pa

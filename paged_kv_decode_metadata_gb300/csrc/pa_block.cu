// Launch of the attention over block-scaled caches (pa_block_mma.cuh), and the join of the
// partial results of several splits.
#include "pa_block_mma.cuh"

namespace pa {
namespace {

constexpr int kJoinThreads = 128;

// A row's pieces combined: M = max m_s, out = sum acc_s e^(m_s - M) / sum l_s e^(m_s - M), lse =
// M + ln of that sum.  The list of a row's pieces is its l values up to the first negative one
// (or num_splits of them); a row whose first l is negative has its output already.  kWarps warps
// take a row's pieces in turn, a lane owning 4 channels; the grid runs over requests and their
// queries, so rows that no request covers are left alone.
template <int kWarps>
__global__ void __launch_bounds__(kJoinThreads) block_join_kernel(const BlockParams p) {
  constexpr int kRows = kJoinThreads / 32 / kWarps;
  __shared__ float4 part[kWarps][32];
  __shared__ float part_l[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % kWarps;
  const int head = blockIdx.x * kRows + warp / kWarps, i = blockIdx.y, b = blockIdx.z;
  const int S = p.num_splits;
  grid_dependency_wait();
  int q_begin = b, q_len = 1;
  if (p.cu_seqlens_q != nullptr) {
    q_begin = p.cu_seqlens_q[b];
    q_len = p.cu_seqlens_q[b + 1] - q_begin;
    if (q_begin < 0 || q_len > p.max_q_len || q_begin > p.total_q - q_len) return;
  }
  if (i >= q_len) return;
  if (kWarps == 1 && head >= p.num_q_heads) return;  // (more warps: one row a block)
  const int64_t row = (static_cast<int64_t>(q_begin) + i) * p.num_q_heads + head;
  const float* m = p.m_out + row * S;
  const float* l = p.l_out + row * S;
  const float4* acc = reinterpret_cast<const float4*>(p.acc_out) + row * S * 32 + lane;
  float top = -CUDART_INF_F, total = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kDeep = 4;
  bool more = true;
  for (int s0 = 0; s0 < S && more; s0 += 32) {
    const float ls = s0 + lane < S ? l[s0 + lane] : -1.f;
    float ms = s0 + lane < S ? m[s0 + lane] : -CUDART_INF_F;
    const uint32_t ends = __ballot_sync(0xffffffffu, ls < 0.f);
    const int count = ends != 0 ? __ffs(ends) - 1 : 32;
    if (s0 == 0 && count == 0) return;  // (every warp of the row alike)
    more = count == 32;
    if (lane >= count) ms = -CUDART_INF_F;
    const float now = fmaxf(top, warp_max(ms));
    const float keep = top == now ? 1.f : expf(top - now);
    total *= keep;
    o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
    // (an empty piece's acc is not written; a NaN score shows in the sum alone)
    const float f = ms == -CUDART_INF_F ? (lane < count && ls != ls ? 1.f : 0.f) : expf(ms - now);
    const float lf = f == 0.f ? 0.f : f * ls;
    for (int s = w; s < count; s += kDeep * kWarps) {
      float4 a[kDeep];
      float fs[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int at = min(s + u * kWarps, count - 1);
        fs[u] = __shfl_sync(0xffffffffu, f, at);
        const float add = __shfl_sync(0xffffffffu, lf, at);
        if (s + u * kWarps >= count) fs[u] = 0.f;
        if (fs[u] != 0.f) {
          a[u] = acc[(s0 + at) * 32];
          total += add;
        }
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (fs[u] != 0.f) {
          o.x = fmaf(fs[u], a[u].x, o.x);
          o.y = fmaf(fs[u], a[u].y, o.y);
          o.z = fmaf(fs[u], a[u].z, o.z);
          o.w = fmaf(fs[u], a[u].w, o.w);
        }
    }
    top = now;
  }
  if constexpr (kWarps > 1) {
    part[w][lane] = o;
    if (lane == 0) part_l[w] = total;
    __syncthreads();
    if (w != 0) return;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    total = 0.f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) {  // (every warp saw all maxima: one reference)
      const float4 a = part[u][lane];
      total += part_l[u];
      o.x += a.x;
      o.y += a.y;
      o.z += a.z;
      o.w += a.w;
    }
  }
  const float inv = total > 0.f || total != total ? 1.f / total : 0.f;
  static_cast<uint2*>(p.out)[row * 32 + lane] =
      make_uint2(mma::pack_bf16(o.x * inv, o.y * inv), mma::pack_bf16(o.z * inv, o.w * inv));
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = top == -CUDART_INF_F && total == total ? top : top + logf(total);
}

}  // namespace

cudaError_t launch_block(const BlockParams& p, int columns, cudaStream_t stream, bool use_pdl) {
  return columns == 8    ? block::launch_one<8>(p, stream, use_pdl)
         : columns == 16 ? block::launch_one<16>(p, stream, use_pdl)
                         : block::launch_one<32>(p, stream, use_pdl);
}

cudaError_t launch_block_join(const BlockParams& p, cudaStream_t stream, bool use_pdl) {
  // up to four pieces are one round of loads of a warp; more are shared out over four warps
  const bool one = p.num_splits <= 4;
  const unsigned heads = static_cast<unsigned>(one ? (p.num_q_heads + 3) / 4 : p.num_q_heads);
  const dim3 grid(heads, static_cast<unsigned>(p.max_q_len), static_cast<unsigned>(p.bs));
  return fail_at(launch_kernel(one ? block_join_kernel<1> : block_join_kernel<4>, grid, dim3(kJoinThreads), 0,
                               stream, use_pdl, p),
                 "cudaLaunchKernelEx (join)");
}

}  // namespace pa

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

// ---- attention --------------------------------------------------------------------------------

constexpr int kWarps = 4;

// One block per (split, query head, query row of the request); a warp takes every fourth
// position, a lane 4 channels.
template <bool kInt8>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const TreeParams p, int page_size) {
  __shared__ float m_s[kWarps], l_s[kWarps];
  __shared__ float4 o_s[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int qi = blockIdx.x;
  const int head = blockIdx.y, b = blockIdx.z;
  const int kvh = head / (p.num_q_heads / p.num_kv_heads);
  grid_dependency_wait();
  const int q_begin = p.cu_seqlens_q[b];
  int q_len = p.cu_seqlens_q[b + 1] - q_begin;
  if (q_begin < 0 || q_len < 0 || q_len > p.max_q_len || q_begin > p.total_q - q_len) {
    if (threadIdx.x == 0 && head == 0 && blockIdx.x == 0) record_error(p.err, kErrSeqLenOutOfRange);
    q_len = 0;
  }
  if (qi >= q_len) return;
  const int cap = p.max_seq_pages * page_size;
  int n = p.cache_seqlens[b];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0 && head == 0 && blockIdx.x == 0) record_error(p.err, kErrSeqLenOutOfRange);
    n = n < 0 ? 0 : cap;
  }
  const int64_t row = static_cast<int64_t>(q_begin) + qi;
  const uint32_t* mask = p.tree_mask + row * (2 * p.mask_words);
  const uint2 qw = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                  (row * p.num_q_heads + head) * 128)[lane];
  const float q0 = bf16_lo(qw.x), q1 = bf16_hi(qw.x), q2 = bf16_lo(qw.y), q3 = bf16_hi(qw.y);
  const int base = n - q_len;
  const int begin = 0, end = n;
  float m = -CUDART_INF_F, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = begin + warp; j < end; j += kWarps) {
    const int t = j - base;
    if (t >= 0 && !((mask[t >> 5] >> (t & 31)) & 1u)) continue;
    const int pg = p.page_table[static_cast<int64_t>(b) * p.page_table_stride + j / page_size];
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) record_error(p.err, kErrPageOutOfRange);
      continue;
    }
    const int64_t r = (static_cast<int64_t>(pg) * p.num_kv_heads + kvh) * page_size + j % page_size;
    float4 k, v;
    if constexpr (kInt8) {
      const uint32_t kw = static_cast<const uint32_t*>(p.k_cache)[r * 32 + lane];
      const uint32_t vw = static_cast<const uint32_t*>(p.v_cache)[r * 32 + lane];
      const float ks = p.k_scale[r], vs = p.v_scale[r];
      s8x4_to_float(kw, k.x, k.y, k.z, k.w);
      s8x4_to_float(vw, v.x, v.y, v.z, v.w);
      k.x *= ks; k.y *= ks; k.z *= ks; k.w *= ks;
      v.x *= vs; v.y *= vs; v.z *= vs; v.w *= vs;
    } else {
      const uint2 kw = static_cast<const uint2*>(p.k_cache)[r * 32 + lane];
      const uint2 vw = static_cast<const uint2*>(p.v_cache)[r * 32 + lane];
      k = make_float4(bf16_lo(kw.x), bf16_hi(kw.x), bf16_lo(kw.y), bf16_hi(kw.y));
      v = make_float4(bf16_lo(vw.x), bf16_hi(vw.x), bf16_lo(vw.y), bf16_hi(vw.y));
    }
    const float x = warp_sum(q0 * k.x + q1 * k.y + q2 * k.z + q3 * k.w) * p.q_scale;
    const float m_new = fmaxf(m, x);
    const float a = exp2f(m - m_new), w = exp2f(x - m_new);
    m = m_new;
    l = l * a + w;
    o.x = o.x * a + w * v.x;
    o.y = o.y * a + w * v.y;
    o.z = o.z * a + w * v.z;
    o.w = o.w * a + w * v.w;
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  o_s[warp][lane] = o;
  __syncthreads();
  if (warp != 0) return;
  float mm = -CUDART_INF_F;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, m_s[w]);
  float total = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = 0; w < kWarps; ++w) {
    const float a = m_s[w] == -CUDART_INF_F ? 0.f : exp2f(m_s[w] - mm);
    const float4 ow = o_s[w][lane];
    total += l_s[w] * a;
    o.x += ow.x * a; o.y += ow.y * a; o.z += ow.z * a; o.w += ow.w * a;
  }
  const int64_t slot = row * p.num_q_heads + head;
  {
    if (p.num_splits > 1 && lane == 0) p.l_out[slot * p.num_splits] = -1.f;
    const float inv = total > 0.f ? 1.f / total : 0.f;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    static_cast<uint2*>(p.out)[slot * 32 + lane] = make_uint2(
        *reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (p.lse != nullptr && lane == 0)
      p.lse[slot] = mm == -CUDART_INF_F ? mm : mm * 0.69314718055994530942f + logf(total);
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
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += 32) {
      const float ls = s0 + lane < S ? l[s0 + lane] : -1.f;
      const uint32_t ends = __ballot_sync(0xffffffffu, ls < 0.f);
      const int count = ends != 0 ? __ffs(ends) - 1 : 32;
      const float ms = lane < count ? m[s0 + lane] : -CUDART_INF_F;
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
    const float inv = top == -CUDART_INF_F ? 0.f : 1.f / total;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    static_cast<uint2*>(p.out)[row * 32 + lane] = make_uint2(
        *reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (p.lse != nullptr && lane == 0)
      p.lse[row] = top == -CUDART_INF_F ? top : top + logf(total);
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

cudaError_t launch_tree(const TreeParams& p, bool int8, int group, int page_size,
                        cudaStream_t stream, bool use_pdl) {
  if (!int8) return launch_tree_mma_bf16(p, group, page_size, stream, use_pdl);
  const dim3 grid(static_cast<unsigned>(p.max_q_len),
                  static_cast<unsigned>(p.num_q_heads), static_cast<unsigned>(p.bs));
  return fail_at(launch_kernel(int8 ? tree_kernel<true> : tree_kernel<false>, grid, dim3(kWarps * 32),
                               0, stream, use_pdl, p, page_size),
                 "cudaLaunchKernelEx");
}

}  // namespace pa

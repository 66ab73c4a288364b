// The attention weights of a decode step added up per cached row.
//
// Mathematics.  w[j] += sum over the G query heads of a kv head of 2^(x_j log2 e - lse log2 e):
// the scores are recomputed from K (half of the cache, read once) and the step's own
// log-sum-exp, so no weight ever passes through memory between the step and this kernel.
//
// Layout.  S = K Q^T on the tensor cores with M = 16 tokens, N = 8 heads, K = 16 channels.
// The contraction order over channels is free, so a lane's share of a row is chosen to be
// 16-byte pieces: piece j of lane tig holds channels 32 j + 8 tig .. + 7 (bf16), its 32
// contiguous bytes the A registers of every k-step (int8; the codes widen exactly to fp16).
// K goes from global memory straight to the
// MMA registers; nothing is staged.  A warp owns 16 tokens at a time.
//
// Bound by memory: K, and the weights read and written.
#include <math_constants.h>

#include "pa_splitk_mma.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kBlockTokens = 256;

template <bool kInt8, int kNT>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const WeightsParams p, int page_size) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int G = p.num_q_heads / p.num_kv_heads;
  grid_dependency_wait();

  const int cap = p.max_seq_pages * page_size;
  int n = p.cache_seqlens[b];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0) record_error(p.err, kErrSeqLenOutOfRange);
    n = n < 0 ? 0 : cap;
  }
  const int begin = blockIdx.x * kBlockTokens, end = min(n, begin + kBlockTokens);
  if (begin >= end) return;

  // Q fragments (B operand) in the channel order of the K pieces, and the scores' factors
  uint32_t qb[kNT][8][2];
  float qf[kNT][2], base[kNT][2];
  if constexpr (kInt8) {
    SplitKParams sp = {};
    sp.q = p.q;
    sp.num_q_heads = p.num_q_heads;
    sp.q_scale = p.q_scale;
    float kbias[kNT][2];  // (of biased codes: not needed here)
    mma::load_q_fragments<true, kNT>(sp, b, 1, kvh, G, gid, tig, qb, kbias, qf);
  } else {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int col = 8 * nt + gid;
      const uint4* row = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(p.q) +
          (static_cast<int64_t>(b) * p.num_q_heads + kvh * G + col) * 128);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 w = col < G ? row[4 * j + tig] : make_uint4(0u, 0u, 0u, 0u);
        qb[nt][2 * j][0] = w.x;
        qb[nt][2 * j][1] = w.y;
        qb[nt][2 * j + 1][0] = w.z;
        qb[nt][2 * j + 1][1] = w.w;
      }
      qf[nt][0] = qf[nt][1] = p.q_scale;
    }
  }
  bool live[kNT][2];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * nt + 2 * tig + e;
      const float lse = col < G ? p.lse[static_cast<int64_t>(b) * p.num_q_heads + kvh * G + col]
                                : -CUDART_INF_F;
      live[nt][e] = lse != -CUDART_INF_F;
      base[nt][e] = lse * 1.4426950408889634f;
    }

  const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.page_table_stride;
  for (int t0 = begin + warp * 16; t0 < end; t0 += kWarps * 16) {
    const int pg = pt[t0 / page_size];
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) record_error(p.err, kErrPageOutOfRange);
      continue;
    }
    const int64_t row0 = (static_cast<int64_t>(pg) * p.num_kv_heads + kvh) * page_size + t0 % page_size;
    float acc[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    float ks[2] = {1.f, 1.f};
    if constexpr (kInt8) {
      const uint4* k0 = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.k_cache) +
                                                       (row0 + gid) * 128) + 2 * tig;
      const uint4 r[4] = {k0[0], k0[1], k0[64], k0[65]};  // rows gid and gid + 8
      ks[0] = p.k_scale[row0 + gid];
      ks[1] = p.k_scale[row0 + gid + 8];
      const uint32_t w0[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
      const uint32_t w1[8] = {r[2].x, r[2].y, r[2].z, r[2].w, r[3].x, r[3].y, r[3].z, r[3].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x0 = w0[j] ^ 0x80808080u, x1 = w1[j] ^ 0x80808080u;
        uint32_t a[4] = {
            mma::biased_bytes_to_f16x2(x0, 0x4140), mma::biased_bytes_to_f16x2(x1, 0x4140),
            mma::biased_bytes_to_f16x2(x0, 0x4342), mma::biased_bytes_to_f16x2(x1, 0x4342)};
        // the codes' +1152 comes off exactly in fp16 (an offset of 1152 sum(q) in the score
        // would cost it about 2^-19)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&a[u]),
                                    __floats2half2_rn(1152.f, 1152.f));
          a[u] = *reinterpret_cast<const uint32_t*>(&v);
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) mma::mma16816<true>(acc[nt], a, qb[nt][j][0], qb[nt][j][1]);
      }
    } else {
      const uint4* k0 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_cache) +
                                                       (row0 + gid) * 128) + tig;
      uint4 r0[4], r1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r0[j] = k0[4 * j];
        r1[j] = k0[4 * j + 128];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo[4] = {r0[j].x, r1[j].x, r0[j].y, r1[j].y};
        const uint32_t hi[4] = {r0[j].z, r1[j].z, r0[j].w, r1[j].w};
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          mma::mma16816<false>(acc[nt], lo, qb[nt][2 * j][0], qb[nt][2 * j][1]);
          mma::mma16816<false>(acc[nt], hi, qb[nt][2 * j + 1][0], qb[nt][2 * j + 1][1]);
        }
      }
    }
    float sum[2] = {0.f, 0.f};  // tokens gid and gid + 8, over this lane's heads
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = acc[nt][i] * qf[nt][i & 1] * ks[i >> 1];
        if (live[nt][i & 1]) sum[i >> 1] += mma::fast_exp2(x - base[nt][i & 1]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    // (an add without a return: rows of a page that requests share meet in the L2)
    if (tig < 2) {
      const int j = t0 + gid + 8 * tig;
      if (j < end) atomicAdd(p.weights + row0 + gid + 8 * tig, tig == 0 ? sum[0] : sum[1]);
    }
  }
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, bool int8, int group, int page_size,
                           cudaStream_t stream, bool use_pdl) {
  const int64_t tokens = static_cast<int64_t>(p.max_seq_pages) * page_size;
  const dim3 grid(static_cast<unsigned>((tokens + kBlockTokens - 1) / kBlockTokens),
                  static_cast<unsigned>(p.num_kv_heads), static_cast<unsigned>(p.bs));
  void (*kernel)(const WeightsParams, int) =
      int8 ? (group > 8 ? weights_kernel<true, 2> : weights_kernel<true, 1>)
           : (group > 8 ? weights_kernel<false, 2> : weights_kernel<false, 1>);
  return fail_at(launch_kernel(kernel, grid, dim3(kWarps * 32), 0, stream, use_pdl, p, page_size),
                 "cudaLaunchKernelEx");
}

}  // namespace pa

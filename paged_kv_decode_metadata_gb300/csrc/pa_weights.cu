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
// Bound by memory: K, and the weights read and written: 64 requests of up to 16K tokens (int8)
// take 104 us (5.7 TB/s), one of 8K (bf16) 3.1 us, which is what an eager launch costs the host.
#include <math_constants.h>

#include "pa_splitk_mma.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

// One warp's 16 tokens of K on their way to the MMA registers: rows gid and gid + 8.
template <bool kInt8>
struct Tile {
  uint4 a[kInt8 ? 2 : 4], b[kInt8 ? 2 : 4];
  float sa, sb;  // int8: their scales

  // row0: the pool row of the first token
  __device__ __forceinline__ void load(const WeightsParams& p, int64_t row0, int gid, int tig) {
    constexpr int kStep = kInt8 ? 1 : 4;  // pieces of a lane: side by side, or every fourth
    const uint4* k0 = static_cast<const uint4*>(p.k_cache) + (row0 + gid) * (kInt8 ? 8 : 16) +
                      (kInt8 ? 2 : 1) * tig;
#pragma unroll
    for (int j = 0; j < (kInt8 ? 2 : 4); ++j) {
      a[j] = k0[kStep * j];
      b[j] = k0[kStep * j + 8 * (kInt8 ? 8 : 16)];
    }
    if constexpr (kInt8) {
      sa = p.k_scale[row0 + gid];
      sb = p.k_scale[row0 + gid + 8];
    }
  }
};

// kRuns: a block has several runs of tokens.
template <bool kInt8, int kNT, bool kRuns>
__global__ void __launch_bounds__(kWarps * 32)
    weights_kernel(const WeightsParams p, int page_shift, int block_tokens) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int G = p.num_q_heads / p.num_kv_heads;
  grid_dependency_wait();

  const int page_size = 1 << page_shift, cap = p.max_seq_pages << page_shift;
  int n = p.cache_seqlens[b];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0) record_error(p.err, kErrSeqLenOutOfRange);
    n = n < 0 ? 0 : cap;
  }
  const int first = blockIdx.x * block_tokens;
  if (first >= n) return;

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
  constexpr int kStep = kWarps * 16;
#pragma unroll 1
  for (int run = first;;) {
    const int end = min(n, run + block_tokens);
    int at = run + warp * 16;
    int next = at < end ? pt[at >> page_shift] : 0;
#pragma unroll 1
    for (; at < end; at += kStep) {
      const int pg = next;
      if (at + kStep < end) next = pt[(at + kStep) >> page_shift];
      if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) record_error(p.err, kErrPageOutOfRange);
        continue;
      }
      const int64_t row0 = ((static_cast<int64_t>(pg) * p.num_kv_heads + kvh) << page_shift) +
                           (at & (page_size - 1));
      Tile<kInt8> k;
      k.load(p, row0, gid, tig);
      float acc[kNT][4];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
      float ks[2] = {1.f, 1.f};
      if constexpr (kInt8) {
        ks[0] = k.sa;
        ks[1] = k.sb;
        const uint32_t w0[8] = {k.a[0].x, k.a[0].y, k.a[0].z, k.a[0].w, k.a[1].x, k.a[1].y, k.a[1].z, k.a[1].w};
        const uint32_t w1[8] = {k.b[0].x, k.b[0].y, k.b[0].z, k.b[0].w, k.b[1].x, k.b[1].y, k.b[1].z, k.b[1].w};
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
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo[4] = {k.a[j].x, k.b[j].x, k.a[j].y, k.b[j].y};
          const uint32_t hi[4] = {k.a[j].z, k.b[j].z, k.a[j].w, k.b[j].w};
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
        const int j = at + gid + 8 * tig;
        if (j < end) atomicAdd(p.weights + row0 + gid + 8 * tig, tig == 0 ? sum[0] : sum[1]);
      }
    }
    if constexpr (!kRuns) return;
    run += static_cast<int>(gridDim.x) * block_tokens;
    if (run >= n) return;
  }
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, bool int8, int group, int page_size,
                           cudaStream_t stream, bool use_pdl) {
  // Tokens of a run: the more the fewer loads of Q (a fifth of the time at 256), but only
  // while the blocks fill every slot (8 per SM) a few times over.  bs64 ragged to 16K int8:
  // 181 / 133 / 112 / 104 / 107 us with 64 / 128 / 256 / 512 / 1024; one request of 8K:
  // 3.5 / 3.5 / 4.5 / 6.7 us with 64 / 128 / 256 / 512.
  const int64_t tokens = static_cast<int64_t>(p.max_seq_pages) * page_size;
  const int64_t units = static_cast<int64_t>(p.num_kv_heads) * p.bs;
  const int64_t usual = tokens < 16384 ? tokens : 16384;
  int block_tokens = 128;
  while (block_tokens < 512 && usual / (2 * block_tokens) * units >= 152 * 8 * 3) block_tokens *= 2;
  // Tables for longer contexts than that: the requests may be short all the same, and a block
  // without work costs 0.6 ns, so the blocks stop at four times the slots (and at what 16K
  // take) and have several runs each.  8K contexts under a table for 1M: one request 5.4 us
  // (13.6 with a block a run; 3.5 under a table for 8K), 32 ragged ones, int8, 32 (270; 30).
  // One run a block has a kernel of its own: the loop cost 1.5 to 10 % there.
  const int64_t runs = (tokens + block_tokens - 1) / block_tokens;
  int64_t most = (152 * 8 * 4 + units - 1) / units;
  if (most < 16384 / block_tokens && block_tokens == 512) most = 16384 / block_tokens;
  const int64_t rounds = (runs + most - 1) / most;
  const dim3 grid(static_cast<unsigned>((runs + rounds - 1) / rounds),
                  static_cast<unsigned>(p.num_kv_heads), static_cast<unsigned>(p.bs));
  const bool wide = group > 8, many = rounds > 1;
  void (*kernel)(const WeightsParams, int, int) =
      many ? (int8 ? (wide ? weights_kernel<true, 2, true> : weights_kernel<true, 1, true>)
                   : (wide ? weights_kernel<false, 2, true> : weights_kernel<false, 1, true>))
           : (int8 ? (wide ? weights_kernel<true, 2, false> : weights_kernel<true, 1, false>)
                   : (wide ? weights_kernel<false, 2, false> : weights_kernel<false, 1, false>));
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  return fail_at(launch_kernel(kernel, grid, dim3(kWarps * 32), 0, stream, use_pdl, p, shift,
                               block_tokens),
                 "cudaLaunchKernelEx");
}

}  // namespace pa

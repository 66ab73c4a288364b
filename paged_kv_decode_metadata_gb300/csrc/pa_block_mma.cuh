// Attention over a block-scaled cache (e4m3 codes, one scale per block of tokens and head) on
// the 5th-generation tensor cores (tcgen05, kind::f8f6f4).
//
// Mathematics.  x_j = s q . K_j, out = sum_j e^(x_j - m) V_j / sum_j e^(x_j - m), one pass with
// a running maximum.  The codes go from memory to the tensor cores as they are, so the other
// operand of each product is e4m3, too, in pieces: a query row, scaled by a power of two, is
// hi + lo / 16, which holds bf16 exactly (8 significant bits are 4 and 4; what is lost of the
// row's small channels is 2^-21 of its largest); a weight is h1 + h2 / 16 + h3 / 256, within
// 2^-12 of itself, or within 2^-26 of the chunk's largest weight times V scale.  Each piece has
// columns of its own in the product, so the pieces are added in fp32.  The K scale multiplies
// the fp32 score; the V scale multiplies the weight before it is cut into pieces, relative to
// the chunk's largest V scale, which multiplies the chunk's product.  Products leave tensor
// memory chunk by chunk and are summed in fp32 registers: no accumulator is rescaled in place,
// and long contexts do not add up the tensor cores' truncation.
//
// Shape.  M is the cache side: scores are S^T = K Q^T (128 tokens x 2 C columns), outputs O^T =
// V^T P^T (128 channels x 3 C), C = 8, 16 or 32 columns of (query, head) pairs of one kv head.
// So few columns cost few cycles, a thread owns a token in the softmax and a channel in the
// sums, and neither K nor V is moved or widened.  A column's maximum goes over 128 threads: a
// warp reduction, four numbers in shared memory, one barrier a chunk.
//   warps 0-3   softmax and sums
//   warp 4      TMA: a ring of 16 KiB tiles, K and V in turn
//   warp 5      issues K Q^T (two score buffers: a chunk ahead of the softmax)
//   warp 6      issues V^T P^T
#pragma once

#include <math_constants.h>

#include "pa_splitk_mma.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace block {

constexpr int kTile = 128;  // tokens of a chunk, channels
constexpr int kTileBytes = kTile * 128;
constexpr int kThreads = 224;
constexpr int kTmaWarp = 4, kScoreWarp = 5, kOutWarp = 6;
constexpr float kLift = 256.f;  // of a chunk's largest weight: its first piece

template <int C>
struct Shape {
  static constexpr int kScoreCols = 2 * C;
  static constexpr int kOutCols = (3 * C + 15) / 16 * 16;
  static constexpr int kTmemCols = 2 * kScoreCols + kOutCols <= 64    ? 64
                                   : 2 * kScoreCols + kOutCols <= 128 ? 128
                                                                      : 256;
  static constexpr int kSlots = C == 8 ? 4 : C == 16 ? 6 : 5;
  static constexpr int kBlocks = C == 8 ? 3 : 2;  // resident per SM
  static constexpr int kRing = 0;
  static constexpr int kQ = kSlots * kTileBytes;
  static constexpr int kP = kQ + kScoreCols * 128;
  static constexpr int kEnd = kP + kOutCols * 128;
  struct alignas(16) Control {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full, s_full[2], s_empty[2], p_full, o_full, drained[2];
    // per warp: a column's largest score, the largest V scale; of even and of odd chunks (a warp
    // may write the next chunk's while another still reads this one's)
    alignas(16) float peak[2][C + 1][4];
    alignas(16) float sum[C][4];
    float factor[C];  // of a column's scores
    uint32_t tmem;
    int abort, issued;
  };
  static constexpr int kBytes = kEnd + static_cast<int>(sizeof(Control)) + 1024;  // + alignment
  static_assert((kBytes + 1024) * kBlocks <= 228 * 1024, "resident blocks");
  static_assert(kTmemCols * kBlocks <= 512, "tensor memory");
};

// Instruction descriptor: fp32 accumulator, e4m3 operands, M = 128.
constexpr uint32_t instruction(int n, bool a_mn_major) {
  return (1u << 4) | (a_mn_major ? 1u << 15 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
         (static_cast<uint32_t>(kTile / 16) << 24);
}

__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                    bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(umma::kOperandHigh), "r"(accumulate ? 1u : 0u)
      : "memory");
}

template <int kCols>
__device__ __forceinline__ void alloc(uint32_t* out) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(out)),
               "n"(kCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int kCols>
__device__ __forceinline__ void dealloc(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(kCols)
               : "memory");
}

// 8 columns of the warp's 32 lanes: thread i gets row i.  Valid after wait_ld.
__device__ __forceinline__ void ld8(uint32_t addr, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
                 "=f"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void wait_ld(float (&a)[8], float (&b)[8], float (&c)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]),
                 "+f"(a[7]), "+f"(b[0]), "+f"(b[1]), "+f"(b[2]), "+f"(b[3]), "+f"(b[4]), "+f"(b[5]),
                 "+f"(b[6]), "+f"(b[7]), "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]), "+f"(c[4]),
                 "+f"(c[5]), "+f"(c[6]), "+f"(c[7])
               :
               : "memory");
}
__device__ __forceinline__ void wait_ld(float (&a)[8], float (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]),
                 "+f"(a[7]), "+f"(b[0]), "+f"(b[1]), "+f"(b[2]), "+f"(b[3]), "+f"(b[4]), "+f"(b[5]),
                 "+f"(b[6]), "+f"(b[7])
               :
               : "memory");
}

// The largest over the warp (a NaN is ignored).
__device__ __forceinline__ float warp_peak(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Two values to e4m3 codes (round to even, saturated), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
// The values of two codes, exactly.
__device__ __forceinline__ float2 from_codes(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int C>
__global__ void __launch_bounds__(kThreads, Shape<C>::kBlocks)
    block_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const BlockParams prm) {
  using Sh = Shape<C>;
  constexpr int kSlots = Sh::kSlots;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const uint32_t base_addr = smem_addr(smem);
  typename Sh::Control& ctl = *reinterpret_cast<typename Sh::Control*>(smem + Sh::kEnd);
  volatile int* abort_flag = &ctl.abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform for the compiler too)
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int S = prm.num_splits;
  const int split = static_cast<int>(blockIdx.x) % S, tile = static_cast<int>(blockIdx.x) / S;
  const int G = prm.group;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.s_empty[i], 4);
      mbar_init(&ctl.drained[i], 1);
    }
    mbar_init(&ctl.p_full, 4);
    mbar_init(&ctl.o_full, 1);
    ctl.abort = 0;
    ctl.issued = 0;
    fence_barrier_init();
  }
  grid_dependency_wait();

  // the request, checked; its queries of this tile and the tokens of this split
  int q_begin = b, q_len = 1;
  if (prm.cu_seqlens_q != nullptr) {
    q_begin = prm.cu_seqlens_q[b];
    q_len = prm.cu_seqlens_q[b + 1] - q_begin;
    if (q_begin < 0 || q_len < 0 || q_len > prm.max_q_len || q_begin > prm.total_q - q_len) {
      if (tid == 0 && blockIdx.x == 0 && kvh == 0) record_error(prm.err, kErrSeqLenOutOfRange);
      q_len = 0;
    }
  }
  int n = prm.cache_seqlens[b];
  const int page_shift = prm.page_shift, P = 1 << page_shift;
  const int cap = prm.max_seq_pages << page_shift;
  if (n < 0 || n > cap) {
    if (tid == 0 && blockIdx.x == 0 && kvh == 0) record_error(prm.err, kErrSeqLenOutOfRange);
    n = n < 0 ? 0 : cap;
  }
  const int q0 = tile * prm.tile_queries;
  const int live = min(q_len - q0, prm.tile_queries);  // queries of this tile
  if (live <= 0) return;
  const int cols = live * G;
  // query i sees positions below n - q_len + i + 1
  const int end = max(0, min(n, n - q_len + q0 + live));
  const int first = min(split * prm.split_chunks * kTile, end);
  const int last = min(end, first + prm.split_chunks * kTile);
  const int chunks = (last - first + kTile - 1) / kTile;
  const int64_t row0 = (static_cast<int64_t>(q_begin) + q0) * prm.num_q_heads + kvh * G;
  auto row_of = [&](int c) { return row0 + static_cast<int64_t>(c / G) * prm.num_q_heads + c % G; };
  if (chunks == 0) {
    for (int c = tid; c < cols; c += kThreads) {
      if (S > 1) {
        prm.m_out[row_of(c) * S + split] = -CUDART_INF_F;
        prm.l_out[row_of(c) * S + split] = 0.f;
      } else if (prm.lse != nullptr) {
        prm.lse[row_of(c)] = -CUDART_INF_F;
      }
    }
    if (S == 1)
      for (int i = tid; i < cols * 16; i += kThreads)
        static_cast<uint4*>(prm.out)[row_of(i >> 4) * 16 + (i & 15)] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }

  if (warp == kScoreWarp) alloc<Sh::kTmemCols>(&ctl.tmem);
  umma::fence_before();
  __syncthreads();  // barriers initialised, tensor memory allocated
  umma::fence_after();
  const uint32_t tmem = ctl.tmem;
  const uint32_t out_col = tmem + 2 * Sh::kScoreCols;
  auto give_up = [&]() {
    record_error(prm.err, kErrWaitTimeout);
    *abort_flag = 1;
  };

  if (warp < 4) {
    // ======================= softmax and sums ============================================
    const uint32_t lane_base = static_cast<uint32_t>(warp) << 21;  // lane 32 warp
    // ----- the query rows' pieces: a warp takes every fourth column, a lane 4 channels -----
    for (int c = warp; c < C; c += 4) {
      uint2 w = make_uint2(0u, 0u);
      if (c < cols)
        w = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(prm.q) + row_of(c) * 128)[lane];
      const float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
      const float big = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
      const int e = big > 0.f ? 7 - mma::float_exponent(big) : 0;  // the largest in [128, 256)
      const float up = mma::pow2_clamped(e);
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float y0 = x[2 * i] * up, y1 = x[2 * i + 1] * up;
        const uint32_t h = to_codes(y0, y1);
        const float2 back = from_codes(h);
        hi |= h << (16 * i);
        lo |= to_codes(16.f * (y0 - back.x), 16.f * (y1 - back.y)) << (16 * i);
      }
      auto at = [&](int row) {
        return smem + Sh::kQ + mma::swz(row, lane >> 2) + 4 * (lane & 3);
      };
      *reinterpret_cast<uint32_t*>(at(c)) = hi;
      *reinterpret_cast<uint32_t*>(at(C + c)) = lo;
      // (an infinite or NaN channel makes the row's scores NaN)
      const bool finite = __all_sync(0xffffffffu, fabsf(x[0]) < CUDART_INF_F && fabsf(x[1]) < CUDART_INF_F &&
                                                      fabsf(x[2]) < CUDART_INF_F && fabsf(x[3]) < CUDART_INF_F);
      if (lane == 0) ctl.factor[c] = finite ? prm.q_scale * mma::pow2_clamped(-e) : CUDART_NAN_F;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mma::mbar_arrive(&ctl.q_full);
    softmax_barrier();

    // ----- scales: a thread's token's, a chunk ahead; its page two chunks ahead -----------
    const int32_t* pt = prm.page_table + static_cast<int64_t>(b) * prm.page_table_stride;
    const int blocks = P >> prm.block_shift;  // of a page
    auto page_of = [&](int i) -> int {
      const int pos = first + i * kTile + tid;
      return pos < last ? pt[pos >> page_shift] : 0;
    };
    auto scale_at = [&](int i, int page) -> int64_t {
      const int row = (first + i * kTile + tid) & (P - 1);
      if (page < 0 || page >= prm.num_pages) page = 0;  // (the TMA warp reports it)
      return (static_cast<int64_t>(page) * prm.num_kv_heads + kvh) * blocks + (row >> prm.block_shift);
    };
    int page = page_of(0);
    float ks = 0.f, vs = 0.f;
    if (first + tid < last) {
      ks = prm.k_scale[scale_at(0, page)];
      vs = prm.v_scale[scale_at(0, page)];
    }
    page = page_of(1);

    float m[C], l[C], acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      m[c] = -CUDART_INF_F;
      l[c] = 0.f;
      acc[c] = 0.f;
    }
    float v_peak = 0.f;  // of the chunk before
    bool ok = true;
    auto add_product = [&](int i) {  // acc += the product of chunk i
      ok = ok && mbar_wait_bounded(&ctl.o_full, i & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      umma::fence_after();
      const float f = v_peak * (1.f / kLift);
#pragma unroll
      for (int g = 0; g < C / 8; ++g) {
        float h1[8], h2[8], h3[8];
        ld8(out_col + lane_base + 8 * g, h1);
        ld8(out_col + lane_base + C + 8 * g, h2);
        ld8(out_col + lane_base + 2 * C + 8 * g, h3);
        wait_ld(h1, h2, h3);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[8 * g + j] = fmaf(fmaf(fmaf(h3[j], 1.f / 16.f, h2[j]), 1.f / 16.f, h1[j]), f, acc[8 * g + j]);
      }
      umma::fence_before();
    };
    for (int i = 0; i < chunks; ++i) {
      const int pos = first + i * kTile + tid;
      // what the next chunks need, on its way
      float ks_next = 0.f, vs_next = 0.f;
      if (pos + kTile < last) {
        ks_next = prm.k_scale[scale_at(i + 1, page)];
        vs_next = prm.v_scale[scale_at(i + 1, page)];
      }
      page = page_of(i + 2);
      // (after a wait that gave up, the chunks that are left only meet the barrier, so that no
      // warp waits there for good)
      ok = ok && mbar_wait_bounded(&ctl.s_full[i & 1], (i >> 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      umma::fence_after();
      const uint32_t sc = tmem + (i & 1) * Sh::kScoreCols + lane_base;
      const int seen0 = n - q_len + q0 + 1;  // positions that the tile's first query sees
      const bool masked = first + (i + 1) * kTile > min(last, seen0);
      // columns 8 g .. of this token; positions past the chunk's end or past the column's
      // query's own are not seen
      auto scores = [&](int g, float (&x)[8]) {
        float lo[8];
        ld8(sc + 8 * g, x);
        ld8(sc + C + 8 * g, lo);
        wait_ld(x, lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(lo[j], 1.f / 16.f, x[j]) * (ctl.factor[8 * g + j] * ks);
        if (masked) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (pos >= last || pos >= seen0 + (8 * g + j) / G) x[j] = -CUDART_INF_F;
        }
      };
      auto scores_done = [&]() {
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mma::mbar_arrive(&ctl.s_empty[i & 1]);
      };
      constexpr bool kKeep = C == 8;  // (wider ones are read again: registers)
      float x[8];
      if (ok) {
#pragma unroll
        for (int g = 0; g < C / 8; ++g) {
          scores(g, x);
          if (kKeep) scores_done();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float top = warp_peak(x[j]);
            if (lane == 0) ctl.peak[i & 1][8 * g + j][warp] = top;
          }
        }
        vs = pos < last ? vs : 0.f;
        const float top = warp_peak(fabsf(vs));
        if (lane == 0) ctl.peak[i & 1][C][warp] = top;
      }
      softmax_barrier();
      if (ok && i > 0) add_product(i - 1);
      if (ok) {
        const float4 t = *reinterpret_cast<const float4*>(ctl.peak[i & 1][C]);
        v_peak = fmaxf(umma::max3(t.x, t.y, t.z), t.w);
        // the scale relative to the chunk's largest (a chunk of zeros: 0)
        const float lift = v_peak > 0.f ? vs / v_peak * kLift : v_peak == 0.f ? 0.f : CUDART_NAN_F;
        unsigned char* p_tile = smem + Sh::kP;
        auto at = [&](int row) { return p_tile + mma::swz(row, tid >> 4) + (tid & 15); };
#pragma unroll
        for (int g = 0; g < C / 8; ++g) {
          if (!kKeep) scores(g, x);
          if (!kKeep && g == C / 8 - 1) scores_done();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = 8 * g + j;
            const float4 t = *reinterpret_cast<const float4*>(ctl.peak[i & 1][c]);
            const float top = fmaxf(umma::max3(t.x, t.y, t.z), fmaxf(t.w, m[c]));
            if (top != m[c]) {  // (all threads alike)
              const float alpha = mma::fast_exp2(m[c] - top);
              m[c] = top;
              acc[c] *= alpha;
              l[c] *= alpha;
            }
            x[j] = mma::fast_exp2(x[j] - (top == -CUDART_INF_F ? 0.f : top));
            l[c] += x[j];
            x[j] *= lift;
          }
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float y0 = x[j], y1 = x[j + 1];
#pragma unroll
            for (int piece = 0; piece < 3; ++piece) {
              const int row = piece * C + 8 * g + j;
              const uint32_t codes = to_codes(y0, y1);
              *at(row) = static_cast<unsigned char>(codes);
              *at(row + 1) = static_cast<unsigned char>(codes >> 8);
              if (piece < 2) {
                const float2 back = from_codes(codes);
                y0 = 16.f * (y0 - back.x);
                y1 = 16.f * (y1 - back.y);
              }
            }
          }
        }
        // V rows past the last token may hold anything, and 0 times NaN is NaN
        const int valid = last - (first + i * kTile);
        if (valid < kTile) {
          const int it = 2 * i + 1, slot = it % kSlots;
          ok = mbar_wait_bounded(&ctl.full[slot], static_cast<uint32_t>(it / kSlots) & 1u);
          ok = __all_sync(0xffffffffu, ok);
          for (int u = valid * 8 + tid; u < kTile * 8 && ok; u += 128)
            *reinterpret_cast<uint4*>(smem + Sh::kRing + slot * kTileBytes + u * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        umma::fence_before();
        __syncwarp();
        if (ok && lane == 0) mma::mbar_arrive(&ctl.p_full);
      }
      ks = ks_next;
      vs = vs_next;
    }
    add_product(chunks - 1);
    if (!ok && lane == 0) give_up();
    // ----- the columns' results -------------------------------------------------------------
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float part = warp_sum(l[c]);
      if (lane == 0) ctl.sum[c][warp] = part;
    }
    softmax_barrier();
    if (ok) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (c >= cols) break;
        const float4 t = *reinterpret_cast<const float4*>(ctl.sum[c]);
        const float total = (t.x + t.y) + (t.z + t.w);
        const int64_t row = row_of(c);
        const float m_nat = m[c] * 0.69314718055994530942f;  // -inf stays -inf
        if (S > 1) {
          prm.acc_out[(row * S + split) * 128 + tid] = acc[c];
          if (tid == 0) {
            prm.m_out[row * S + split] = m_nat;
            prm.l_out[row * S + split] = total;
          }
        } else {
          const float inv = total > 0.f || total != total ? 1.f / total : 0.f;
          static_cast<__nv_bfloat16*>(prm.out)[row * 128 + tid] = __float2bfloat16_rn(acc[c] * inv);
          if (prm.lse != nullptr && tid == 0)
            prm.lse[row] = m[c] == -CUDART_INF_F && total == total ? m[c] : m_nat + logf(total);
        }
      }
    }
    umma::fence_before();
  } else if (warp == kTmaWarp) {
    // ======================= TMA ==========================================================
    const int box_shift = min(page_shift, 6), box_rows = 1 << box_shift;
    const int boxes_of_tile = kTile >> box_shift;  // of a tile: a lane issues one
    const int32_t* pt = prm.page_table + static_cast<int64_t>(b) * prm.page_table_stride;
    const uint64_t policy = l2_evict_first_policy();
    auto page_of = [&](int i) -> int {
      const int pos = first + i * kTile + lane * box_rows;
      return lane < boxes_of_tile && pos < last ? pt[pos >> page_shift] : -1;
    };
    int next = page_of(0);
    bool ok = true;
    for (int i = 0; i < chunks && ok; ++i) {
      const int pos = first + i * kTile + lane * box_rows;
      const bool mine = lane < boxes_of_tile && pos < last;
      int page = next;
      next = i + 1 < chunks ? page_of(i + 1) : -1;
      if (mine && (page < 0 || page >= prm.num_pages)) {
        record_error(prm.err, kErrPageOutOfRange);
        page = 0;
      }
      const int boxes = min(boxes_of_tile, (last - first - i * kTile + box_rows - 1) >> box_shift);
      for (int kv = 0; kv < 2; ++kv) {
        const int it = 2 * i + kv, slot = it % kSlots;
#ifdef PA_TIMESTAMPS
        // failure-detection test of the instrumented build: after three tiles nothing is issued,
        // so the other warps' waits give up with products in flight
        if (prm.hold_loads && it >= 3) continue;
#endif
        ok = it < kSlots || mbar_wait_bounded(&ctl.empty[slot], static_cast<uint32_t>(it / kSlots - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (lane == 0) {
          ctl.issued = it + 1;
          mbar_arrive_expect_tx(&ctl.full[slot], boxes * box_rows * 128);
        }
        __syncwarp();
        if (mine)
          mma::tma_load_4d(base_addr + Sh::kRing + slot * kTileBytes + lane * box_rows * 128,
                           kv ? &map_v : &map_k, 0, pos & (P - 1), kvh, page, &ctl.full[slot], policy);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == kScoreWarp) {
    // ======================= K Q^T ========================================================
    if (umma::elect()) {
      constexpr uint32_t kDesc = instruction(Sh::kScoreCols, false);
      const uint32_t q = umma::operand(base_addr + Sh::kQ, 16);
      bool ok = mbar_wait_bounded(&ctl.q_full, 0);
      for (int i = 0; i < chunks && ok; ++i) {
        const int it = 2 * i, slot = it % kSlots;
        ok = mbar_wait_bounded(&ctl.full[slot], static_cast<uint32_t>(it / kSlots) & 1u);
        if (ok && i >= 2) ok = mbar_wait_bounded(&ctl.s_empty[i & 1], ((i >> 1) - 1) & 1u);
        if (!ok) break;
        umma::fence_after();
        const uint32_t k = umma::operand(base_addr + Sh::kRing + slot * kTileBytes, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma(tmem + (i & 1) * Sh::kScoreCols, k + 2 * j, q + 2 * j, kDesc, j > 0);
        umma::commit(&ctl.empty[slot]);
        umma::commit(&ctl.s_full[i & 1]);
      }
      if (!ok) {
        give_up();
        umma::commit(&ctl.drained[0]);  // what was issued must be over before the memory is freed
        mbar_wait_bounded(&ctl.drained[0], 0);
      }
    }
    __syncwarp();
  } else if (warp == kOutWarp) {
    // ======================= V^T P^T ======================================================
    if (umma::elect()) {
      constexpr uint32_t kDesc = instruction(Sh::kOutCols, true);
      const uint32_t p = umma::operand(base_addr + Sh::kP, 16);
      bool ok = true;
      for (int i = 0; i < chunks && ok; ++i) {
        const int it = 2 * i + 1, slot = it % kSlots;
        ok = mbar_wait_bounded(&ctl.full[slot], static_cast<uint32_t>(it / kSlots) & 1u);
        if (ok) ok = mbar_wait_bounded(&ctl.p_full, i & 1u);
        if (!ok) break;
        umma::fence_after();
        // 32 tokens a step: 4 KiB of V, 32 bytes of a row of P
        const uint32_t v = umma::operand(base_addr + Sh::kRing + slot * kTileBytes, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma(out_col, v + j * (4096 >> 4), p + 2 * j, kDesc, j > 0);
        umma::commit(&ctl.empty[slot]);
        umma::commit(&ctl.o_full);
      }
      if (!ok) {
        give_up();
        umma::commit(&ctl.drained[1]);
        mbar_wait_bounded(&ctl.drained[1], 0);
      }
    }
    __syncwarp();
  }
  trigger_dependents();
  umma::fence_before();
  __syncthreads();  // every load from tensor memory is over
  if (*abort_flag && tid == 0) {
    // copies in flight must land before the block's memory is given up
    const int issued = *static_cast<volatile int*>(&ctl.issued);
    for (int i = max(0, issued - kSlots); i < issued; ++i)
      mbar_wait_bounded(&ctl.full[i % kSlots], static_cast<uint32_t>(i / kSlots) & 1u);
  }
  if (warp == kScoreWarp) {
    umma::fence_after();
    dealloc<Sh::kTmemCols>(tmem);
  }
}

// ---- host side ------------------------------------------------------------------------------

template <int C>
cudaError_t launch_one(const BlockParams& p, int tiles, cudaStream_t stream, bool use_pdl) {
  CUtensorMap mk, mv;
  cudaError_t e = mma::encode_pool_map(&mk, p.k_cache, true, p.num_pages, p.num_kv_heads, 1 << p.page_shift);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (K)");
  e = mma::encode_pool_map(&mv, p.v_cache, true, p.num_pages, p.num_kv_heads, 1 << p.page_shift);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (V)");
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(block_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<C>::kBytes);
    if (e != cudaSuccess) return fail_at(e, "shared-memory attribute");
    configured.fetch_or(bit);
  }
  return fail_at(launch_kernel(block_kernel<C>,
                               dim3(static_cast<unsigned>(p.num_splits * tiles), p.num_kv_heads, p.bs),
                               dim3(kThreads), static_cast<size_t>(Shape<C>::kBytes), stream, use_pdl, mk, mv, p),
                 "cudaLaunchKernelEx");
}

}  // namespace block
}  // namespace pa

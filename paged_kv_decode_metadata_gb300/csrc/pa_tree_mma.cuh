// Tree attention on the 5th-generation tensor cores (tcgen05).
//
// Mathematics.  The G heads of a kv head and the q_len drafted tokens of a request are
// q_len * G rows over the same keys: per kv head S = Q K^T and O += P V are dense products of
// M = 128 rows, 128 tokens and 128 channels.  Softmax is one pass over the tokens: a row's
// weights are 2^(x - r) for a reference r that moves only when a score passes it by more
// than 2^8, so the accumulator is rescaled a few times per split, not per chunk.  Weights
// enter P V rounded to bf16 (2^-8 of each weight's share); their sum l stays unrounded fp32.
//
// Shape of a block.  One CTA per SM takes up to 256 rows (two tiles of 128) of one (request,
// kv head) over one split, so a K/V chunk of 128 tokens is fetched once for both.  Two
// streams, each with a score buffer and an accumulator in tensor memory (4 x 128 columns =
// all 512): with two tiles a stream is a tile; with one, the streams take alternate chunks
// and are joined at the end.  So the tensor cores work on one stream while the other's
// softmax runs.
//   warps 0-3, 4-7   softmax of stream 0, 1: a thread owns a row, so maxima and sums need no
//                    exchange; scores come from and weights go back to tensor memory (P
//                    takes the place of S, as the A operand of P V)
//   warp 8           TMA: a ring of five 32 KiB tiles, K and V in turn; a lane issues one
//                    box (up to 64 tokens of one page, 64 channels), so small pages cost no
//                    more time than large ones
//   warp 9           one thread issues every MMA: P V of chunk c, then Q K^T of the stream's
//                    next chunk, whose scores are ready when the other stream's are used up
//   warps 10, 11     zero the V rows past the request's last token (0 * NaN is NaN)
// Masks cost nothing before the last chunks: only chunks that reach the drafted positions
// look at the ancestor bits.
//
// Bound by: memory up to about 256 rows per kv head (64 KiB of K/V per 128 tokens against
// 1024 tensor cycles per tile), the tensor cores above.
#pragma once

#include "pa_splitk_mma.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace tree {

constexpr int kTile = 128;            // rows of a tile, tokens of a chunk
constexpr int kSoftmaxThreads = 256;  // two groups of four warps
constexpr int kTmaWarp = 8, kMmaWarp = 9, kFixWarp = 10;
constexpr int kThreads = 384;
// registers per thread after the split: 256 x 224 + 128 x 56 = 384 x 168 at launch
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");
constexpr int kSlots = 5;             // ring tiles
constexpr int kHalfBytes = kTile * 128;       // 64 channels of 128 rows
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kMergeStride = 132;     // floats; the pad spreads a column over the banks

struct Shared {
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kEnd = kRing + kSlots * kTileBytes;
  struct Control {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full, s_full[2], p_half[2], p_ready[2], o_full[2], v_last, v_fixed, drained;
    uint32_t tmem;
    int abort, issued;
  };
  static constexpr int kBytes = kEnd + static_cast<int>(sizeof(Control)) + 1024;  // + alignment
};
static_assert(Shared::kBytes <= 227 * 1024, "one block's shared memory");
static_assert(kTile * kMergeStride * 4 + 2 * kTile * 8 <= kSlots * kTileBytes, "join buffer");

// Bits of the 32 positions from p0 that a row sees: every committed one (< base), of the
// drafted ones those of its mask (bit t: position base + t), none at or past `end`.
__device__ __forceinline__ uint32_t visible(int p0, int base, int end, const uint32_t* mask,
                                            int words) {
  const int left = end - p0, t = p0 - base;
  if (left <= 0) return 0u;
  uint32_t bits;
  if (t <= -32) {
    bits = 0xffffffffu;
  } else if (t < 0) {
    bits = (mask[0] << -t) | ((1u << -t) - 1u);
  } else {
    const int w = t >> 5;
    const uint32_t lo = w < words ? mask[w] : 0u, hi = w + 1 < words ? mask[w + 1] : 0u;
    bits = __funnelshift_r(lo, hi, t & 31);
  }
  return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

template <int P>
__global__ void __launch_bounds__(kThreads, 1)
    tree_mma_kernel(const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const TreeParams prm, int pairs) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base_addr = smem_addr(smem);
  Shared::Control& ctl = *reinterpret_cast<Shared::Control*>(smem + Shared::kEnd);
  volatile int* abort_flag = &ctl.abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = prm.num_q_heads / prm.num_kv_heads;
  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y / pairs, pair = blockIdx.y - kvh * pairs;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.q_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.s_full[s], 1);
      mbar_init(&ctl.p_half[s], 4);
      mbar_init(&ctl.p_ready[s], 4);
      mbar_init(&ctl.o_full[s], 1);
    }
    mbar_init(&ctl.v_last, 1);
    mbar_init(&ctl.v_fixed, 2);
    mbar_init(&ctl.drained, 1);
    ctl.abort = 0;
    ctl.issued = 0;
    fence_barrier_init();
  }
  grid_dependency_wait();

  // ---- the block's rows and tokens (every thread computes them alike) --------------------
  const int q_begin = prm.cu_seqlens_q[b];
  int q_len = prm.cu_seqlens_q[b + 1] - q_begin;
  if (q_begin < 0 || q_len < 0 || q_len > prm.max_q_len || q_begin > prm.total_q - q_len) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) record_error(prm.err, kErrSeqLenOutOfRange);
    q_len = 0;
  }
  const int cap = prm.max_seq_pages * P;
  int n = prm.cache_seqlens[b];
  if (n < 0 || n > cap) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) record_error(prm.err, kErrSeqLenOutOfRange);
    n = n < 0 ? 0 : cap;
  }
  const int rows = min(q_len * G - pair * 2 * kTile, 2 * kTile);  // of this block
  if (rows <= 0) return;
  const bool two = rows > kTile;  // two tiles: a stream each
  const int base = n - q_len;
  const int begin = split * prm.pages_per_split * P;
  const int end = min(n, begin + prm.pages_per_split * P);
  const int n_tok = end - begin;
  const int S = prm.num_splits;
  // output slot of row r of tile t (the row's query and head)
  auto slot_of = [&](int t, int r) -> int64_t {
    const int row = (pair * 2 + t) * kTile + r;
    const int qi = row / G;
    return (static_cast<int64_t>(q_begin) + qi) * prm.num_q_heads + kvh * G + (row - qi * G);
  };

  if (n_tok <= 0) {  // nothing to attend to in this split
    trigger_dependents();
    for (int r = tid; r < rows; r += kThreads) {
      const int64_t slot = slot_of(0, r);
      if (S > 1) {
        prm.m_out[slot * S + split] = -CUDART_INF_F;
        prm.l_out[slot * S + split] = 0.f;
      } else if (prm.lse != nullptr) {
        prm.lse[slot] = -CUDART_INF_F;
      }
    }
    if (S == 1) {
      for (int i = tid; i < rows * 16; i += kThreads)
        static_cast<uint4*>(prm.out)[slot_of(0, i >> 4) * 16 + (i & 15)] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }

  if (warp == kMmaWarp) umma::alloc_all(&ctl.tmem);
  umma::fence_before();
  __syncthreads();  // barriers initialised, tensor memory allocated
  umma::fence_after();
  const uint32_t tmem = ctl.tmem;
  // columns: scores (and weights) of stream s at 128 s, accumulator at 256 + 128 s
  auto s_col = [&](int s) { return tmem + static_cast<uint32_t>(s) * kTile; };
  auto o_col = [&](int s) { return tmem + 256u + static_cast<uint32_t>(s) * kTile; };

  const int chunks = (n_tok + kTile - 1) / kTile;
  const int last_valid = n_tok - (chunks - 1) * kTile;  // tokens of the last chunk
  // a partial last chunk: its V tile completes v_last, is cleaned, and is handed on by v_fixed
  const bool clean_last = last_valid < kTile;
  // chunks of stream s: all of them (two tiles), or every second one from s
  auto stream_chunks = [&](int s) { return two ? chunks : (chunks + 1 - s) / 2; };
  auto give_up = [&]() {
    record_error(prm.err, kErrWaitTimeout);
    *abort_flag = 1;
  };

  if (warp < kTmaWarp) {
    // ======================= softmax ===================================================
    umma::registers_up<kSoftmaxRegs>();
    const int s = warp >> 2, r = tid & (kTile - 1);
    const int tile = two ? s : 0;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 (warp % 4)
    const uint32_t sc = s_col(s) + lane_base, oc = o_col(s) + lane_base;
    const int row = (pair * 2 + tile) * kTile + r;
    const bool live = row < q_len * G;
    const uint32_t* mask = prm.tree_mask + (static_cast<int64_t>(q_begin) + (live ? row / G : 0)) *
                                               (2 * prm.mask_words);
    const int words = 2 * prm.mask_words;
    const float scale = prm.q_scale;
    const int mine = stream_chunks(s);
    float m_ref = -CUDART_INF_F, l = 0.f;  // the row's reference and sum of weights
    for (int k = 0; k < mine; ++k) {
      const int c = two ? k : 2 * k + s;
      const int p0 = begin + c * kTile;
      if (!mbar_wait_bounded(&ctl.s_full[s], static_cast<uint32_t>(k) & 1u)) {
        if (lane == 0) give_up();
        break;
      }
      umma::fence_after();
      const bool tail = p0 + kTile > min(base, end);  // drafted or missing positions
      float x[kTile];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t(&v)[32] = *reinterpret_cast<uint32_t(*)[32]>(&x[32 * i]);
        umma::ld32(sc + 32 * i, v);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) umma::wait_ld(*reinterpret_cast<uint32_t(*)[32]>(&x[32 * i]));
      if (tail) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t bits = live ? visible(p0 + 32 * i, base, end, mask, words) : 0u;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            x[32 * i + j] = (bits >> j) & 1u ? x[32 * i + j] : -CUDART_INF_F;
        }
        __syncwarp();
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int j = 4; j < kTile - 4; j += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = umma::max3(mx[u], x[j + u], x[j + 4 + u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], x[kTile - 4 + u]);
      // (sm_scale > 0: the largest score is the largest product)
      const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      float alpha = 1.f;
      if (m_new > m_ref + mma::kMaxSlack) {
        alpha = m_ref == -CUDART_INF_F ? 0.f : mma::fast_exp2(m_ref - m_new);
        m_ref = m_new;
        l *= alpha;
      }
      __syncwarp();
      // the accumulator follows a moved reference (before the first product there is none)
      if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[32];
          umma::ld32(oc + 32 * i, o);
          umma::wait_ld(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
          umma::st32(oc + 32 * i, o);
        }
      }
      const float ref = m_ref == -CUDART_INF_F ? 0.f : m_ref;
      const uint64_t scale2 = umma::pair(scale, scale), ref2 = umma::pair(-ref, -ref);
      uint64_t sum[4] = {0, 0, 0, 0};  // pairs of +0
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float lo, hi;
          umma::unpair(umma::fma2(umma::pair(x[32 * i + 2 * j], x[32 * i + 2 * j + 1]), scale2, ref2),
                       lo, hi);
          lo = mma::fast_exp2(lo);
          hi = mma::fast_exp2(hi);
          sum[j & 3] = umma::add2(sum[j & 3], umma::pair(lo, hi));
          w[j] = mma::pack_bf16(lo, hi);
        }
        umma::st16(sc + 16 * i, w);
        if (i == 1) {  // half of the weights: their products may start
          umma::wait_st();
          umma::fence_before();
          __syncwarp();
          if (lane == 0) mma::mbar_arrive(&ctl.p_half[s]);
        }
      }
      float lo, hi;
      umma::unpair(umma::add2(umma::add2(sum[0], sum[1]), umma::add2(sum[2], sum[3])), lo, hi);
      l += lo + hi;
      umma::wait_st();
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mma::mbar_arrive(&ctl.p_ready[s]);
    }

    // ----- the rows' results -----------------------------------------------------------
    const bool has = mine > 0;
    if (has && !*abort_flag && !mbar_wait_bounded(&ctl.o_full[s], 0) && lane == 0) give_up();
    umma::fence_after();
    trigger_dependents();
    float factor = 1.f;  // of this stream's accumulator
    float* joined = reinterpret_cast<float*>(smem + Shared::kRing);
    float2* ml = reinterpret_cast<float2*>(joined + kTile * kMergeStride);
    // (both streams' products are over before either writes into the ring)
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (!two) {  // one tile: join the streams, stream 1 hands its rows over
      ml[s * kTile + r] = make_float2(m_ref, l);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float2 other = ml[(1 - s) * kTile + r];
      const float m_all = fmaxf(m_ref, other.x);
      if (m_all != -CUDART_INF_F) {
        factor = m_ref == -CUDART_INF_F ? 0.f : mma::fast_exp2(m_ref - m_all);
        l = l * factor + (other.x == -CUDART_INF_F ? 0.f : other.y * mma::fast_exp2(other.x - m_all));
        m_ref = m_all;
      }
      if (s == 1 && has) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[32];
          umma::ld32(oc + 32 * i, o);
          umma::wait_ld(o);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            joined[r * kMergeStride + 32 * i + j] = __uint_as_float(o[j]) * factor;
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    const bool add = !two && stream_chunks(1) > 0;
    const bool write = live && !*abort_flag;
    if (two || s == 0) {
      const int64_t slot = write ? slot_of(tile, r) : 0;
      const float inv = S == 1 ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      factor *= inv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[32];
        umma::ld32(oc + 32 * i, o);
        umma::wait_ld(o);
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          y[j] = __uint_as_float(o[j]) * factor;
          if (add) y[j] += joined[r * kMergeStride + 32 * i + j] * inv;
        }
        if (write && S == 1) {
          uint4* out = static_cast<uint4*>(prm.out) + slot * 16 + 4 * i;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            out[j] = make_uint4(mma::pack_bf16(y[8 * j], y[8 * j + 1]),
                                mma::pack_bf16(y[8 * j + 2], y[8 * j + 3]),
                                mma::pack_bf16(y[8 * j + 4], y[8 * j + 5]),
                                mma::pack_bf16(y[8 * j + 6], y[8 * j + 7]));
        } else if (write) {
          float4* acc = reinterpret_cast<float4*>(prm.acc_out) + (slot * S + split) * 32 + 8 * i;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
        __syncwarp();
      }
      if (write) {
        const float m_nat = m_ref * 0.69314718055994530942f;  // -inf stays -inf
        if (S > 1) {
          prm.m_out[slot * S + split] = m_nat;
          prm.l_out[slot * S + split] = l;
        } else if (prm.lse != nullptr) {
          prm.lse[slot] = m_ref == -CUDART_INF_F ? m_ref : m_nat + logf(l);
        }
      }
    }
    umma::fence_before();
  } else {
    umma::registers_down<kOtherRegs>();
    if (warp == kTmaWarp) {
    // ======================= TMA ========================================================
    constexpr int kBoxRows = P < 64 ? P : 64;
    constexpr int kBoxes = kTile / kBoxRows;
    const uint64_t policy = l2_evict_first_policy();
    if (lane == 0) {
      const int tiles = two ? 2 : 1;
      mbar_arrive_expect_tx(&ctl.q_full, tiles * kTileBytes);
      for (int t = 0; t < tiles; ++t)
        for (int h = 0; h < 2; ++h)
          asm volatile(
              "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
              " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(base_addr + Shared::kQ + t * kTileBytes +
                                                     h * kHalfBytes),
              "l"(reinterpret_cast<uint64_t>(&map_q)), "r"(64 * h), "r"(kvh * G),
              "r"(q_begin + (pair * 2 + t) * (kTile / G)), "r"(smem_addr(&ctl.q_full))
              : "memory");
    }
    // lane -> (box of the chunk, channel half)
    const int box = lane >> 1, half = lane & 1;
    const int32_t* pt = prm.page_table + static_cast<int64_t>(b) * prm.page_table_stride;
    auto page_of = [&](int c) -> int {  // this lane's page of chunk c, -1: nothing to load
      const int tok = c * kTile + box * kBoxRows;
      return box < kBoxes && tok < n_tok ? pt[(begin + tok) / P] : -1;
    };
    int next = page_of(0);
    bool ok = true;
    for (int c = 0; c < chunks && ok; ++c) {
      const int tok = c * kTile + box * kBoxRows;
      const bool mine = box < kBoxes && tok < n_tok;
      int pg = next;
      if (c + 1 < chunks) next = page_of(c + 1);
      if (mine && (pg < 0 || pg >= prm.num_pages)) {
        record_error(prm.err, kErrPageOutOfRange);
        pg = 0;
      }
      const int boxes = min(kBoxes, (n_tok - c * kTile + kBoxRows - 1) / kBoxRows);
      for (int kv = 0; kv < 2; ++kv) {
        const int i = 2 * c + kv, slot = i % kSlots;
        if (i >= kSlots &&
            (!mbar_wait_bounded(&ctl.empty[slot], static_cast<uint32_t>(i / kSlots - 1) & 1u) ||
             *abort_flag)) {
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) give_up();
          break;
        }
        uint64_t* bar = kv && c == chunks - 1 && clean_last ? &ctl.v_last : &ctl.full[slot];
        if (lane == 0) {
          ctl.issued = i + 1;
          mbar_arrive_expect_tx(bar, boxes * kBoxRows * 256);
        }
        __syncwarp();
        if (mine)
          mma::tma_load_4d(base_addr + Shared::kRing + slot * kTileBytes + half * kHalfBytes +
                               box * kBoxRows * 128,
                           kv ? &map_v : &map_k, 64 * half, (begin + tok) % P, kvh, pg, bar, policy);
        __syncwarp();
      }
    }
  } else if (warp == kMmaWarp) {
    // ======================= MMA issue ==================================================
    if (lane == 0) {
      constexpr uint32_t kScores = umma::instruction(kTile, kTile, false);
      constexpr uint32_t kOutput = umma::instruction(kTile, kTile, true);
      auto tile_addr = [&](int i) { return base_addr + Shared::kRing + (i % kSlots) * kTileBytes; };
      auto wait_tile = [&](int i) {
        return mbar_wait_bounded(&ctl.full[i % kSlots], static_cast<uint32_t>(i / kSlots) & 1u);
      };
      auto scores = [&](int s, int c) {  // S_s = Q_tile K_c^T
        const uint32_t q = base_addr + Shared::kQ + (two ? s : 0) * kTileBytes;
        const uint32_t k = tile_addr(2 * c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t off = (j >> 2) * kHalfBytes + (j & 3) * 32;
          umma::mma_ss(s_col(s), umma::operand(q + off, 16), umma::operand(k + off, 16), kScores, j > 0);
        }
        umma::commit(&ctl.s_full[s]);
      };
      bool ok = mbar_wait_bounded(&ctl.q_full, 0);
      // the first scores of both streams
      for (int s = 0; s < 2 && ok; ++s) {
        if (stream_chunks(s) == 0) break;
        const int c = two ? 0 : s;
        if (s == 0 || !two) ok = wait_tile(2 * c);
        if (!ok) break;
        umma::fence_after();
        scores(s, c);
        if (s == 1 || !two) umma::commit(&ctl.empty[(2 * c) % kSlots]);
      }
      uint32_t used[2] = {0, 0};  // chunks of each stream whose P V has been issued
      for (int c = 0; c < chunks && ok; ++c) {
        const int s_begin = two ? 0 : c & 1, s_end = two ? 2 : s_begin + 1;
        for (int s = s_begin; s < s_end && ok; ++s) {
          ok = mbar_wait_bounded(&ctl.p_half[s], used[s] & 1u);
          if (ok && s == s_begin) {
            ok = c == chunks - 1 && clean_last ? mbar_wait_bounded(&ctl.v_fixed, 0)
                                               : wait_tile(2 * c + 1);
          }
          if (!ok) break;
          umma::fence_after();
          const uint32_t v = tile_addr(2 * c + 1);
          // 16 tokens a step: 8 columns of P, 16 rows of V
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma::mma_ts(o_col(s), s_col(s) + 8 * j, umma::operand(v + j * 16 * 128, kHalfBytes),
                         kOutput, used[s] > 0 || j > 0);
          ok = mbar_wait_bounded(&ctl.p_ready[s], used[s] & 1u);
          if (!ok) break;
          umma::fence_after();
#pragma unroll
          for (int j = 4; j < 8; ++j)
            umma::mma_ts(o_col(s), s_col(s) + 8 * j, umma::operand(v + j * 16 * 128, kHalfBytes),
                         kOutput, true);
          ++used[s];
          if (s == s_end - 1) umma::commit(&ctl.empty[(2 * c + 1) % kSlots]);
          const int next = two ? c + 1 : c + 2;
          if (next < chunks) {
            if (s == s_begin) ok = wait_tile(2 * next);
            if (!ok) break;
            umma::fence_after();
            scores(s, next);
            if (s == s_end - 1) umma::commit(&ctl.empty[(2 * next) % kSlots]);
          } else {
            umma::commit(&ctl.o_full[s]);
          }
        }
      }
      if (!ok) {
        give_up();
        umma::commit(&ctl.drained);  // what was issued must be over before the memory is freed
        mbar_wait_bounded(&ctl.drained, 0);
      }
    }
    __syncwarp();
  } else if (clean_last) {
    // ======================= V rows past the last token ===================================
    const int slot = (2 * chunks - 1) % kSlots;
    if (mbar_wait_bounded(&ctl.v_last, 0)) {
      unsigned char* v = smem + Shared::kRing + slot * kTileBytes;
      for (int u = last_valid * 8 + (warp - kFixWarp) * 32 + lane; u < kTile * 8; u += 64) {
        *reinterpret_cast<uint4*>(v + u * 16) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(v + kHalfBytes + u * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mma::mbar_arrive(&ctl.v_fixed);
    } else if (lane == 0) {
      give_up();
    }
    }
  }

  __syncthreads();  // every load from tensor memory is over
  if (*abort_flag && tid == 0) {
    // copies in flight must land before the block's memory is given up
    const int issued = *static_cast<volatile int*>(&ctl.issued);
    for (int i = max(0, issued - kSlots); i < issued; ++i) {
      if (i == 2 * chunks - 1 && clean_last) {
        mbar_wait_bounded(&ctl.v_last, 0);
      } else {
        mbar_wait_bounded(&ctl.full[i % kSlots], static_cast<uint32_t>(i / kSlots) & 1u);
      }
    }
    mbar_wait_bounded(&ctl.q_full, 0);
  }
  if (warp == kMmaWarp) {
    umma::fence_after();
    umma::dealloc_all(tmem);
  }
}

// ---- host side ------------------------------------------------------------------------------

// Tensor map over q [total_q, Hq, 128]: a box is 64 channels of the G heads of 128 / G queries.
inline cudaError_t encode_q_map(CUtensorMap* map, const TreeParams& p, int group) {
  mma::EncodeTiledFn encode = mma::encode_tiled_fn();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(p.num_q_heads),
                              static_cast<cuuint64_t>(p.total_q)};
  const cuuint64_t strides[2] = {256, 256 * static_cast<cuuint64_t>(p.num_q_heads)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(kTile / group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int P>
cudaError_t launch_one(const TreeParams& p, int group, cudaStream_t stream, bool use_pdl) {
  CUtensorMap mq, mk, mv;
  cudaError_t e = encode_q_map(&mq, p, group);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (Q)");
  e = mma::encode_pool_map(&mk, p.k_cache, false, p.num_pages, p.num_kv_heads, P);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (K)");
  e = mma::encode_pool_map(&mv, p.v_cache, false, p.num_pages, p.num_kv_heads, P);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (V)");
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(tree_mma_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shared::kBytes);
    if (e != cudaSuccess) return fail_at(e, "shared-memory attribute");
    configured.fetch_or(bit);
  }
  const int pairs = (group * p.max_q_len + 2 * kTile - 1) / (2 * kTile);
  const dim3 grid(static_cast<unsigned>(p.num_splits), static_cast<unsigned>(p.num_kv_heads * pairs),
                  static_cast<unsigned>(p.bs));
  return fail_at(launch_kernel(tree_mma_kernel<P>, grid, dim3(kThreads),
                               static_cast<size_t>(Shared::kBytes), stream, use_pdl, mq, mk, mv, p,
                               pairs),
                 "cudaLaunchKernelEx");
}

}  // namespace tree
}  // namespace pa

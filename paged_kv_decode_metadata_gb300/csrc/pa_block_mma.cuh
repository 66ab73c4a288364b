// Attention over a block-scaled cache (e4m3 codes, one scale per block of tokens and head) on
// the 5th-generation tensor cores (tcgen05, kind::f8f6f4).
//
// Mathematics.  x_j = s q . K_j, out = sum_j e^(x_j - m) V_j / sum_j e^(x_j - m), one pass with
// a running maximum.  The codes go from memory to the tensor cores as they are, so the other
// operand of each product has 8 bits, too, in pieces.  A query row, scaled by a power of two, is
// hi + lo / 16 in e4m3, which holds bf16 exactly (8 significant bits are 4 and 4; what is lost of the
// row's small channels is 2^-21 of its largest).  A weight, e^(x - m) times the V scale, the chunk's
// largest V scale lifted to [2^14, 2^15), is rounded to fp16 (2^-11 of itself) and is
// h1 + h2 + (h3 + h4) / 128 in e5m2, which is the upper byte of an fp16: 3 bits a piece, 12 in all.
// e5m2 for its range, since weights are as small as scores lie apart: they are exact from 2^-13 up, and
// what is lost of smaller ones is 2^-23 + 2^-25, 2^-36 of the largest scale's weight of 1 (three pieces
// in e4m3 end 2^-25 below it: beside a token 18 above the others, those were gone).  Pieces of one scale
// are added up by the product, the others in fp32 registers.  The K scale multiplies the
// fp32 score; what lifts the V scales is undone on the chunk's product.  Products leave tensor
// memory chunk by chunk and are summed in fp32 registers: no accumulator is rescaled in place,
// and long contexts do not add up the tensor cores' truncation.
//
// Shape.  M is the cache side: scores are S^T = K Q^T (128 tokens x 2 C columns), outputs O^T =
// V^T P^T (128 channels x 2 C, two passes; C = 8: 4 C), C = 8, 16 or 32 columns of (query, head)
// pairs of one kv head.  So few columns cost few cycles, a thread owns a token in the softmax and a channel in the
// sums, and neither K nor V is moved or widened.  Four warps have 8 columns; a column's maximum
// goes over their 128 threads: a warp reduction, four numbers in shared memory, one barrier a
// chunk.
//   warps 0 .. C/2 - 1   softmax and sums, four for each 8 columns
//   then one each        TMA: a ring of 16 KiB tiles, K and V in turn, running ahead into the
//                        next piece; K Q^T (two score buffers: a chunk ahead of the softmax);
//                        V^T P^T; the scales, which arrive together with a chunk's scores (so
//                        that the softmax warps neither find them nor wait for them)
// One warp, TMA's, walks the block's share and hands its pieces to the others: code that runs once a
// piece comes from beyond the instruction caches, so there is little of it.
// A unit of work is a tile of columns of one (request, kv head).  The batch's units are laid end
// to end in chunks of 128 tokens and cut into equal shares, one for each of the blocks that are
// resident at once: ragged batches leave none idle, and only units that a cut falls into need
// partials.
//
// Bound by memory with 8 columns: 32 requests of 8192 tokens, 32 / 8 heads, 83 us and 6.4 TB/s; 64
// ragged ones up to 16K, 64 / 8 heads, 161 us and 6.7 TB/s.  With 16 and 32 columns by the softmax
// warps' instructions: 1.35 us a chunk of 32 columns on an SM (16 requests of 8192 tokens, 25 columns: 77
// us, where memory would take 40; 73 with weights of three e4m3 pieces, which lost small ones; of those with
// the scales found by the softmax warps 92, with every warp walking for itself 82).  A column for each
// of the four pieces took 79.5, and 153 in place of 148 us for 32 requests and 32 columns.  One request
// of 1024 tokens: 8.4 us, launches and dependent latencies; short contexts by the same latencies once a unit (256 requests of 128 tokens: 28 us, memory 10).
#pragma once

#include <math_constants.h>

#include "pa_splitk_mma.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace block {

constexpr int kTile = 128;  // tokens of a chunk, channels
constexpr int kTileBytes = kTile * 128;
constexpr float kNothing = -3.402823466e38f;  // a maximum before any score (which, finite, is not below it)

// One piece of work: chunks [c0, c1) of one unit (a tile of queries of a request, a kv head).
struct Piece {
  int b, q_begin, q_len, n;  // the request, its query rows, its cached tokens
  int kvh, tile;
  int c0, c1;
  int slot, pieces;  // which of the unit's pieces this is, and how many it has
};

// A piece as the walking warp hands it to the others: tokens [first, last) of request b, of which the
// tile's first query sees those below `seen` (query i: i more).
struct alignas(16) Job {
  int first, last, seen, cols;  // (0 columns: there are no more pieces)
  int b, kvh, slot, pieces;
  long long row0;  // the first column's row of q and of the results
};

// The batch as one line, unit after unit (by request, kv head, tile), a place for each chunk and
// kUnitCost before them for what a unit costs beside them: block i takes [i share, (i + 1) share),
// or, where units are not cut, the units that start there.  (The host keeps the line's length within
// 31 bits.)
// (Measured at 0 / 1 / 2 / 4: 64 ragged requests to 16K, 64 / 8 heads, 196 / 175 / 174 / 174 us; 8 ragged
// chains to 4001 36 / 31 / 24 / 24 us.)
constexpr int kUnitCost = 2;
struct Walk {
  int b, q_begin, q_len, n, tiles, chunks;  // the request at hand
  int from, kvh, tile;                      // the unit at hand: its first chunk on the line
  int pos, end, share;                      // where the walk is
  int cut;                                  // whether units are cut

  // Lengths of request r as they stand, then checked; `report` records what is wrong with them.
  __device__ __forceinline__ void fetch(const BlockParams& prm, int r) {
    b = r;
    q_begin = r;
    q_len = 1;
    if (prm.cu_seqlens_q != nullptr) {
      q_begin = prm.cu_seqlens_q[r];
      q_len = prm.cu_seqlens_q[r + 1];
    }
    n = prm.cache_seqlens[r];
  }
  __device__ __forceinline__ void check(const BlockParams& prm, bool report) {
    if (prm.cu_seqlens_q != nullptr) {
      q_len -= q_begin;
      if (q_begin < 0 || q_len < 0 || q_len > prm.max_q_len || q_begin > prm.total_q - q_len) {
        if (report) record_error(prm.err, kErrSeqLenOutOfRange);
        q_len = 0;
      }
    }
    const int cap = prm.max_seq_pages << prm.page_shift;
    if (n < 0 || n > cap) {
      if (report) record_error(prm.err, kErrSeqLenOutOfRange);
      n = n < 0 ? 0 : cap;
    }
    // (a division only where there can be several tiles)
    tiles = prm.max_q_len <= prm.tile_queries ? (q_len > 0) : (q_len + prm.tile_queries - 1) / prm.tile_queries;
    chunks = (n + kTile - 1) / kTile;
  }
  __device__ __forceinline__ void load(const BlockParams& prm, int r, bool report) {
    fetch(prm, r);
    check(prm, report);
  }
  __device__ __forceinline__ int length(const BlockParams& prm) const {
    return chunks > 0 ? tiles * prm.num_kv_heads * (chunks + kUnitCost) : 0;
  }

  // Whole-warp: finds the block's share.  Returns whether some request has queries but nothing
  // cached (its rows are no work, but have a result).  A lane has 4 requests of each 128 (one of 32
  // in small batches), whose lengths are asked for at once.
  __device__ __forceinline__ bool start(const BlockParams& prm, int lane) {
    constexpr int kPer = 4;
    const int per = prm.bs <= 32 ? 1 : kPer, round_size = 32 * per;
    Walk r[kPer];
    int total = 0, longest = 0, shortest = INT_MAX, w = 0, incl = 0;
    bool empties = false;
    auto round = [&](int r0, bool report) {
      w = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (k < per) r[k].fetch(prm, min(r0 + lane * per + k, prm.bs - 1));
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (k < per) r[k].check(prm, report);
        if (k >= per || r0 + lane * per + k >= prm.bs) r[k].n = r[k].q_len = r[k].tiles = r[k].chunks = 0;
        w += r[k].length(prm);
      }
      incl = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
    };
    for (int r0 = 0; r0 < prm.bs; r0 += round_size) {
      round(r0, blockIdx.x == 0);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        empties = empties || (r[k].q_len > 0 && r[k].n == 0);
        if (r[k].tiles > 0 && r[k].chunks > 0) {
          longest = max(longest, r[k].chunks);
          shortest = min(shortest, r[k].chunks);
        }
      }
      total += __shfl_sync(0xffffffffu, incl, 31);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    shortest = __reduce_min_sync(0xffffffffu, shortest);
    empties = __any_sync(0xffffffffu, empties);
    // A unit of c > 1 chunks (its places in a row) meets at most floor((c - 2) / share) + 2 shares: a
    // share of (longest - 1) / (num_splits - 1), rounded up, keeps every unit's pieces within num_splits.
    const int S = prm.num_splits, grid = static_cast<int>(gridDim.x);
    share = (total + grid - 1) / grid;
    // Units of one length that fill the blocks well enough stay whole: partials and their join cost
    // more than up to a fifth of a share left idle (256 units of 64 chunks on 304 blocks 82 us whole,
    // 85.5 cut; 512 of them 163 and 161).
    const int unit_places = longest + kUnitCost;
    cut = S > 1 && !(longest == shortest && (total / unit_places + grid - 1) / grid * unit_places <= share + share / 5);
    if (cut && S < longest) share = max(share, (longest + S - 2) / (S - 1));
    const long long at_ll = static_cast<long long>(blockIdx.x) * share;
    pos = static_cast<int>(min(at_ll, static_cast<long long>(total)));
    end = static_cast<int>(min(at_ll + share, static_cast<long long>(total)));
    if (pos >= end) return empties;
    // the request that holds pos
    int before = 0;
    for (int r0 = 0; r0 < prm.bs; r0 += round_size) {
      if (prm.bs > round_size) round(r0, false);
      const uint32_t has = __ballot_sync(0xffffffffu, pos < before + incl);
      if (has != 0) {
        const int lane_of = __ffs(has) - 1;
        int first = before + incl - w;  // (of that lane, whose requests hold pos)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int length_k = r[k].length(prm);
          if (first <= pos && pos < first + length_k) {
            b = r[k].b;
            q_begin = r[k].q_begin;
            q_len = r[k].q_len;
            n = r[k].n;
            tiles = r[k].tiles;
            chunks = r[k].chunks;
            from = first;
          }
          first += length_k;
        }
        b = __shfl_sync(0xffffffffu, b, lane_of);
        q_begin = __shfl_sync(0xffffffffu, q_begin, lane_of);
        q_len = __shfl_sync(0xffffffffu, q_len, lane_of);
        n = __shfl_sync(0xffffffffu, n, lane_of);
        tiles = __shfl_sync(0xffffffffu, tiles, lane_of);
        chunks = __shfl_sync(0xffffffffu, chunks, lane_of);
        from = __shfl_sync(0xffffffffu, from, lane_of);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int places = chunks + kUnitCost;
    int unit = (pos - from) / places;
    if (!cut && unit * places < pos - from) ++unit;  // units that start here
    from += unit * places;
    if (!cut) pos = from;
    from += kUnitCost;
    kvh = tiles == 1 ? unit : unit / tiles;  // (one past the last: the next request)
    tile = unit - kvh * tiles;
    return empties;
  }

  // (No division but for units that a cut falls into: between pieces the block waits for it.)
  __device__ __forceinline__ bool next(const BlockParams& prm, Piece& p) {
    while (pos < end) {
      if (pos >= from + chunks) {  // on to the next unit
        from += chunks + kUnitCost;
        if (++tile == tiles) {
          tile = 0;
          ++kvh;
        }
      }
      if (kvh == prm.num_kv_heads) {  // of the next request that has work
        const int at = from - kUnitCost;
        do {
          load(prm, b + 1, false);
        } while (length(prm) == 0);
        from = at + kUnitCost;
        kvh = tile = 0;
      }
      p.b = b;
      p.q_begin = q_begin;
      p.q_len = q_len;
      p.n = n;
      p.kvh = kvh;
      p.tile = tile;
      p.c0 = max(pos - from, 0);
      p.c1 = cut ? min(chunks, end - from) : chunks;
      p.slot = 0;
      p.pieces = 1;
      if (cut && (p.c0 > 0 || p.c1 < chunks)) {
        const int first = from / share;
        p.slot = static_cast<int>(blockIdx.x) - first;
        p.pieces = (from + chunks - 1) / share - first + 1;
      }
      pos = from + p.c1;
      if (cut && p.c1 < chunks) pos = end;
      if (p.c1 > p.c0) return true;  // (a share may end before a unit's first chunk)
    }
    return false;
  }
};

template <int C>
struct Shape {
  static constexpr int kSoftmaxWarps = C / 2;
  static constexpr int kTmaWarp = kSoftmaxWarps, kScoreWarp = kTmaWarp + 1, kOutWarp = kTmaWarp + 2;
  static constexpr int kScaleWarp = kTmaWarp + 3;
  static constexpr int kThreads = 32 * (kScaleWarp + 1);  // (a warpgroup of these)
  // registers a thread: of the launch, then of the softmax warps and the others
  static constexpr int kLaunchRegs = C == 8 ? 128 : C == 16 ? 80 : 96;
  static constexpr int kSoftmaxRegs = C == 8 ? 168 : C == 16 ? 96 : 104, kOtherRegs = C == 8 ? 80 : C == 16 ? 48 : 64;
  static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + 4 * kOtherRegs) <= kThreads * kLaunchRegs, "register split");
  static constexpr int kScoreCols = 2 * C;
  // The weights' pieces h1 and h3 of a group of 8 columns lie next to one another, and h2 and h4.  h1 and h2
  // have one scale, and h3 and h4: one product adds them up in two passes over V, each with a tile of its
  // own.  (Rows of 16 bytes, which 8 columns would have, are another layout: they take one pass.)
  static constexpr int kPasses = C == 8 ? 1 : 2;
  static constexpr int kOutCols = 4 * C / kPasses;
  static constexpr int kTmemCols = C == 8 ? 64 : C == 16 ? 128 : 256;
  static_assert(2 * kScoreCols + kOutCols <= kTmemCols, "tensor memory");
  static constexpr int kJobs = 4;  // pieces handed over and not yet taken by every warp
  // Tiles in flight: 8 an SM stream best (12 and 6: 64 requests of 16K 329 and 317-321 us against 314-316),
  // and two blocks of them with four rather than three with two.
  static constexpr int kSlots = C <= 16 ? 4 : 10;
  // A slot holds K tiles or V tiles, never both in turn: only then has whoever waits for a tile
  // seen the slot's one before, and a barrier's parity tells which of the two has landed.
  static_assert(kSlots % 2 == 0, "K and V slots");
  static constexpr int kBlocks = C <= 16 ? 2 : 1;  // resident per SM
  static constexpr int kRing = 0;
  static constexpr int kQ = kSlots * kTileBytes;
  static constexpr int kP = kQ + kScoreCols * 128;
  // The weights' tiles, one a pass: a row per token ("MN-major"), rows of 32 or 64 bytes with that swizzle.
  static constexpr int kRowBytes = kOutCols, kWeightsTile = kTile * kRowBytes;
  static constexpr int kStage = kP + kPasses * kWeightsTile;  // the columns' sums on their way out
  static constexpr int kEnd = kStage + C * 128 * 4;
  // High word of their descriptors: the stride offset steps 8 rows; version 1; the swizzle's code.
  static constexpr uint32_t kWeightsHigh = (8u * kRowBytes >> 4) | (1u << 14) | ((kRowBytes == 32 ? 6u : 4u) << 29);
  // Byte offset from kP of a group's pieces in row `t`: h1 and h3 (half 0), h2 and h4 (half 1).
  static __device__ __forceinline__ uint32_t weights_at(int t, int half, int group) {
    const int tile = kPasses == 1 ? 0 : half, c = kPasses == 1 ? half : group;
    return static_cast<uint32_t>(tile * kWeightsTile + t * kRowBytes +
                                 ((c ^ (kRowBytes == 32 ? t >> 2 & 1 : t >> 1 & 3)) << 4));
  }
  struct alignas(16) Control {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full, s_full[2], s_empty[2], p_full, o_full, drained[2];
    // per warp of four: a column's largest score; of even and of odd chunks (a warp may write the next
    // chunk's while another still reads this one's)
    alignas(16) float peak[2][C / 8][4][8];
    // a chunk's scales, K's and V's, block by block, V's times the power of two that brings the largest of
    // them to [2^14, 2^15) (all NaN where it is infinite); and what undoes that
    alignas(16) float2 scales[2][kTile / 16];
    float v_down[2];
    alignas(16) float sum[C][4];
    float inverse[C];
    alignas(16) float factor[C];  // of a column's scores
    Job jobs[kJobs];
    uint64_t job_full[kJobs], job_empty[kJobs];
    uint32_t tmem;
    int abort, issued, empties;
  };
  static constexpr int kBytes = kEnd + static_cast<int>(sizeof(Control)) + 1024;  // + alignment
  static_assert((kBytes + 1024) * kBlocks <= 228 * 1024 && kBytes <= 227 * 1024, "resident blocks");
  static_assert(kTmemCols * kBlocks <= 512, "tensor memory");
};

// Instruction descriptors: fp32 accumulator, M = 128; scores e4m3 by e4m3, products e4m3 by e5m2 with both
// operands "MN-major".
constexpr uint32_t instruction(int n, bool product) {
  return (1u << 4) | (product ? 1u << 10 | 3u << 15 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
         (static_cast<uint32_t>(kTile / 16) << 24);
}

__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t idesc,
                                    bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(umma::kOperandHigh), "r"(b_high), "r"(accumulate ? 1u : 0u)
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
__device__ __forceinline__ void wait_ld(float (&a)[8], float (&b)[8], float (&c)[8], float (&d)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]), "+f"(a[7]),
                 "+f"(b[0]), "+f"(b[1]), "+f"(b[2]), "+f"(b[3]), "+f"(b[4]), "+f"(b[5]), "+f"(b[6]), "+f"(b[7]),
                 "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]), "+f"(c[4]), "+f"(c[5]), "+f"(c[6]), "+f"(c[7]),
                 "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]), "+f"(d[4]), "+f"(d[5]), "+f"(d[6]), "+f"(d[7])
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

// Upper bytes of four fp16 values, e5m2 codes; and what they leave of two of them (exact).
__device__ __forceinline__ uint32_t upper_bytes(uint32_t w01, uint32_t w23) { return __byte_perm(w01, w23, 0x7531); }
__device__ __forceinline__ uint32_t rest_of(uint32_t w) {
  const uint32_t upper = w & 0xff00ff00u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&upper));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t times_128(uint32_t w) {
  const __half2 d = __hmul2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(128.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// (a predicate, not a branch around the arrival)
__device__ __forceinline__ void arrive_if(uint64_t* bar, bool yes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(yes ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ float pick(const float (&x)[8], int i) {
  float y = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) y = i == j ? x[j] : y;
  return y;
}

// The four warps of 8 columns.  (Numbers that the compiler knows: for others it sets all 16 of a
// block's barriers aside.)
template <int kGroups>
__device__ __forceinline__ void group_barrier(int group) {
  if (kGroups == 1 || group == 0) {
    asm volatile("bar.sync 1, 128;" ::: "memory");
  } else if (kGroups == 2 || group == 1) {
    asm volatile("bar.sync 2, 128;" ::: "memory");
  } else if (group == 2) {
    asm volatile("bar.sync 3, 128;" ::: "memory");
  } else {
    asm volatile("bar.sync 4, 128;" ::: "memory");
  }
}

// Whether `yes` holds in all of their threads.
template <int kBarrier>
__device__ __forceinline__ bool barrier_all(bool yes) {
  uint32_t all = yes;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %0, 0;\n\t"
      "bar.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "+r"(all)
      : "n"(kBarrier)
      : "memory");
  return all != 0;
}
template <int kGroups>
__device__ __forceinline__ bool group_all(int group, bool yes) {
  if (kGroups == 1 || group == 0) return barrier_all<1>(yes);
  if (kGroups == 2 || group == 1) return barrier_all<2>(yes);
  return group == 2 ? barrier_all<3>(yes) : barrier_all<4>(yes);
}

template <int C>
__global__ void __launch_bounds__(Shape<C>::kThreads, Shape<C>::kBlocks)
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
  const int S = prm.num_splits, G = prm.group;
  const int page_shift = prm.page_shift, P = 1 << page_shift;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.q_full, Sh::kSoftmaxWarps);
    mbar_init(&ctl.p_full, Sh::kSoftmaxWarps);
    mbar_init(&ctl.o_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 2);  // the scores and the scales
      mbar_init(&ctl.s_empty[i], Sh::kSoftmaxWarps);
      mbar_init(&ctl.drained[i], 1);
    }
    for (int i = 0; i < Sh::kJobs; ++i) {
      mbar_init(&ctl.job_full[i], 1);
      mbar_init(&ctl.job_empty[i], Sh::kSoftmaxWarps + 3);
    }
    ctl.abort = 0;
    ctl.issued = 0;
    fence_barrier_init();
  }
  if (warp == Sh::kScoreWarp) alloc<Sh::kTmemCols>(&ctl.tmem);
  if (warp == Sh::kTmaWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
  }
  umma::fence_before();
  __syncthreads();  // barriers initialised, tensor memory allocated
  umma::fence_after();
  const uint32_t tmem = ctl.tmem;
  const uint32_t out_col = tmem + 2 * Sh::kScoreCols;
  grid_dependency_wait();

  // The TMA warp finds the block's share and goes on.
  Walk walk;
  if (warp == Sh::kTmaWarp) {
    const bool empties = walk.start(prm, lane);
    if (lane == 0) ctl.empties = empties;
    __syncwarp();
    asm volatile("bar.arrive 5, %0;" ::"n"(Sh::kThreads) : "memory");
  } else {
    asm volatile("bar.sync 5, %0;" ::"n"(Sh::kThreads) : "memory");
    if (ctl.empties) {  // requests with queries and an empty cache
      const int at = tid < Sh::kTmaWarp * 32 ? tid : tid - 32;
      constexpr int kOthers = Sh::kThreads - 32;
      Walk w;
      for (int r = blockIdx.x; r < prm.bs; r += gridDim.x) {
        w.load(prm, r, false);
        if (w.n > 0) continue;
        const int64_t first = static_cast<int64_t>(w.q_begin) * prm.num_q_heads;
        const int64_t rows = static_cast<int64_t>(w.q_len) * prm.num_q_heads;
        for (int64_t i = at; i < rows; i += kOthers) {
          if (prm.lse != nullptr) prm.lse[first + i] = -CUDART_INF_F;
          if (S > 1) prm.l_out[(first + i) * S] = -1.f;
        }
        for (int64_t i = at; i < rows * 16; i += kOthers)
          static_cast<uint4*>(prm.out)[first * 16 + i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  auto give_up = [&]() {
    record_error(prm.err, kErrWaitTimeout);
    *abort_flag = 1;
  };
  auto chunks_of = [&](const Job& w) { return (w.last - w.first + kTile - 1) / kTile; };
  // The next piece, for a warp that is not TMA's (`lone`: for one of its threads).  False where the wait for
  // it gave up.
  uint32_t taken = 0;
  auto take = [&](Job& w, bool lone) {
    const uint32_t s = taken % Sh::kJobs;
    bool got = mbar_wait_bounded(&ctl.job_full[s], (taken / Sh::kJobs) & 1u);
    if (!lone) got = __all_sync(0xffffffffu, got);
    if (!got) return false;
    w = ctl.jobs[s];
    if (!lone) __syncwarp();
    arrive_if(&ctl.job_empty[s], lone || lane == 0);
    ++taken;
    return true;
  };

  if (warp < Sh::kSoftmaxWarps) {
    // ======================= softmax and sums ============================================
    umma::registers_up<Sh::kSoftmaxRegs>();
    const int group = warp >> 2, token = tid & 127, w4 = warp & 3;  // 8 columns, a row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(w4) << 21;     // lane 32 (warp % 4)
    uint32_t step = 0;  // chunks of the pieces before
    bool ok = true;
    // of the thread's token in the weights' tiles
    const uint32_t weights_at[2] = {Sh::kP + Sh::weights_at(token, 0, group), Sh::kP + Sh::weights_at(token, 1, group)};
    const int block = token >> prm.block_shift;  // the token's scale of a chunk
    // the queries of the group's columns, a byte each (no division in the loops)
    uint32_t queries[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) queries[j >> 2] |= static_cast<uint32_t>((8 * group + j) / G) << (8 * (j & 3));
    auto query_of = [&](int j) { return static_cast<int>((j & 4 ? queries[1] : queries[0]) >> (8 * (j & 3)) & 0xffu); };
    Job p;
    while (true) {
      // (all warps of a group go on or none does: none may wait for another that has gone; and the sums of the
      // piece before have been read)
      const bool got = group_all<C / 8>(group, take(p, false));
      ok = ok && got;
      if (!got || p.cols == 0) break;
      const int first = p.first, last = p.last, seen0 = p.seen;
      const int chunks = chunks_of(p);
      const int cols = p.cols;
      auto row_of = [&](int j) {  // of column 8 group + j
        return p.row0 + static_cast<int64_t>(query_of(j)) * (prm.num_q_heads - G) + 8 * group + j;
      };
      // ----- the query rows' pieces: a warp has two columns, a lane 4 channels ----------------
      uint2 rows[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = 2 * warp + u;
        rows[u] = c < cols && chunks > 0
                      ? reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(prm.q) + row_of(2 * w4 + u) * 128)[lane]
                      : make_uint2(0u, 0u);
      }
      if (chunks > 0) {
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          const int c = 2 * warp + u;
          const uint2 row = u == 0 ? rows[0] : rows[1];
          const float x[4] = {bf16_lo(row.x), bf16_hi(row.x), bf16_lo(row.y), bf16_hi(row.y)};
          const float mine = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
          const float big = warp_peak(mine);
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
          auto at = [&](int row) { return smem + Sh::kQ + mma::swz(row, lane >> 2) + 4 * (lane & 3); };
          *reinterpret_cast<uint32_t*>(at(c)) = hi;
          *reinterpret_cast<uint32_t*>(at(C + c)) = lo;
          // (an infinite or NaN channel makes the row's scores NaN)
          const bool finite = __all_sync(0xffffffffu, fabsf(x[0]) < CUDART_INF_F && fabsf(x[1]) < CUDART_INF_F &&
                                                          fabsf(x[2]) < CUDART_INF_F && fabsf(x[3]) < CUDART_INF_F);
          if (lane == 0) ctl.factor[c] = finite ? prm.q_scale * mma::pow2_clamped(-e) : CUDART_NAN_F;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        arrive_if(&ctl.q_full, lane == 0);
        group_barrier<C / 8>(group);  // the group's factors
      }

      // Columns that the tile leaves empty (short drafts among longer ones, groups that do not fill
      // it): their four warps only keep the barriers' count, a chunk at a time, and leave the issue
      // slots to the others.  What their columns of the products hold is of no use.
      if (C > 8 && 8 * group >= cols) {
        for (int i = 0; i < chunks; ++i, ++step) {
          const uint32_t buf = step & 1u;
          ok = ok && mbar_wait_bounded(&ctl.s_full[buf], (step >> 1) & 1u);
          ok = __all_sync(0xffffffffu, ok);
          arrive_if(&ctl.s_empty[buf], ok && lane == 0);
          arrive_if(&ctl.p_full, ok && lane == 0);
          ok = ok && mbar_wait_bounded(&ctl.o_full, step & 1u);
          ok = __all_sync(0xffffffffu, ok);
        }
        continue;
      }

      // (two columns an instruction wherever there is one: the schedulers are what bounds 16 and 32
      // columns)
      float m[8], m_mine = kNothing;  // (lane j of eight has column j's once more)
      uint64_t l2[4], acc2[4];
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = kNothing;
#pragma unroll
      for (int k = 0; k < 4; ++k) l2[k] = acc2[k] = umma::pair(0.f, 0.f);
      const uint64_t sixteenth = umma::pair(1.f / 16.f, 1.f / 16.f), small = umma::pair(1.f / 128.f, 1.f / 128.f);
      float v_down = 0.f;  // of the chunk before: what undoes its V scales' power of two
      auto add_product = [&](uint32_t at) {  // acc += the product of chunk `at`
        ok = ok && mbar_wait_bounded(&ctl.o_full, at & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        umma::fence_after();
        float h1[8], h3[8];  // of h1 + h2, of h3 + h4
        const uint32_t oc = out_col + lane_base + 16 * group;
        ld8(oc, h1);
        ld8(oc + 8, h3);
        if constexpr (Sh::kPasses == 1) {
          float h2[8], h4[8];
          ld8(oc + 16, h2);
          ld8(oc + 24, h4);
          wait_ld(h1, h2, h3, h4);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h1[j] += h2[j];
            h3[j] += h4[j];
          }
        } else {
          wait_ld(h1, h3);
        }
        const uint64_t down = umma::pair(v_down, v_down);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = 2 * k;
          const uint64_t sum = umma::fma2(umma::pair(h3[j], h3[j + 1]), small, umma::pair(h1[j], h1[j + 1]));
          acc2[k] = umma::fma2(sum, down, acc2[k]);
        }
        umma::fence_before();
      };
      for (int i = 0;; ++i, ++step) {
        const uint32_t buf = step & 1u;
        float x[8], lift = 0.f, down = 0.f;
        if (i < chunks) {
          const int pos = first + i * kTile + token;
          // (after a wait that gave up, the chunks that are left only meet the barriers, so that no
          // warp waits there for good)
          ok = ok && mbar_wait_bounded(&ctl.s_full[buf], (step >> 1) & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            umma::fence_after();
            const uint32_t sc = tmem + buf * Sh::kScoreCols + lane_base + 8 * group;
            float lo[8];
            ld8(sc, x);
            ld8(sc + C, lo);
            const float2 kv = ctl.scales[buf][block];
            const float ks = kv.x;
            lift = pos < last ? kv.y : 0.f;
            down = ctl.v_down[buf];
            wait_ld(x, lo);
            umma::fence_before();
            __syncwarp();
            arrive_if(&ctl.s_empty[buf], lane == 0);
            const uint64_t ks2 = umma::pair(ks, ks);
            const ulonglong2* factors = reinterpret_cast<const ulonglong2*>(ctl.factor + 8 * group);
            const ulonglong2 f01 = factors[0], f23 = factors[1];
            const uint64_t f[4] = {f01.x, f01.y, f23.x, f23.y};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = 2 * k;
              const uint64_t y = umma::fma2(umma::pair(lo[j], lo[j + 1]), sixteenth, umma::pair(x[j], x[j + 1]));
              umma::unpair(umma::mul2(y, umma::mul2(f[k], ks2)), x[j], x[j + 1]);
            }
            // positions past the chunk's end or past the column's query's own are not seen
            if (first + (i + 1) * kTile > min(last, seen0)) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (pos >= last || pos >= seen0 + query_of(j)) x[j] = -CUDART_INF_F;
            }
            // (all eight at once: with a store behind each they took 665 cycles, not 200)
            float top[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) top[j] = warp_peak(x[j]);
            if (lane == 0) {
              float4* at = reinterpret_cast<float4*>(ctl.peak[buf][group][w4]);
              at[0] = make_float4(top[0], top[1], top[2], top[3]);
              at[1] = make_float4(top[4], top[5], top[6], top[7]);
            }
          }
          group_barrier<C / 8>(group);
        }
        // the product before, which has had the time of a softmax (behind the weights, with two
        // buffers of both, it was slower: 78 us against 73 for 25 columns, 96 against 88 for 10, with the
        // weights cut into three pieces)
        if (i > 0) add_product(step - 1);
        if (i == chunks) break;
        if (ok) {
          // (lane j of eight looks after column j)
          const float* tm = &ctl.peak[buf][group][0][lane & 7];
          const float top = fmaxf(umma::max3(tm[0], tm[8], tm[16]), fmaxf(tm[24], m_mine));
          v_down = down;
          if (__any_sync(0xffffffffu, top != m_mine)) {  // (all threads of the group alike)
            m_mine = top;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float m0 = __shfl_sync(0xffffffffu, top, 2 * k), m1 = __shfl_sync(0xffffffffu, top, 2 * k + 1);
              const uint64_t alpha = umma::pair(mma::fast_exp2(m[2 * k] - m0), mma::fast_exp2(m[2 * k + 1] - m1));
              m[2 * k] = m0;
              m[2 * k + 1] = m1;
              acc2[k] = umma::mul2(acc2[k], alpha);
              l2[k] = umma::mul2(l2[k], alpha);
            }
          }
          const uint64_t lift2 = umma::pair(lift, lift), minus = umma::pair(-1.f, -1.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = 2 * k;
            float d0, d1;  // x - m
            umma::unpair(umma::fma2(umma::pair(m[j], m[j + 1]), minus, umma::pair(x[j], x[j + 1])), d0, d1);
            const uint64_t e2 = umma::pair(mma::fast_exp2(d0), mma::fast_exp2(d1));
            l2[k] = umma::add2(l2[k], e2);
            umma::unpair(umma::mul2(e2, lift2), x[j], x[j + 1]);
          }
          // rounded to fp16 (11 bits), then cut into pieces of 3 bits, the last one rounded
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = mma::pack_f16(x[2 * j], x[2 * j + 1]);
          uint32_t h[4][2];
#pragma unroll
          for (int piece = 0; piece < 4; ++piece) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (piece > 0) w[j] = rest_of(w[j]);
              if (piece == 2) w[j] = times_128(w[j]);  // (below 2^9 before)
              if (piece == 3) w[j] += 0x00800080u;     // (half a step; NaN is in the other pieces)
            }
            h[piece][0] = upper_bytes(w[0], w[1]);
            h[piece][1] = upper_bytes(w[2], w[3]);
          }
          *reinterpret_cast<uint4*>(smem + weights_at[0]) = make_uint4(h[0][0], h[0][1], h[2][0], h[2][1]);
          *reinterpret_cast<uint4*>(smem + weights_at[1]) = make_uint4(h[1][0], h[1][1], h[3][0], h[3][1]);
          // V rows past the last token may hold anything, and 0 times NaN is NaN
          const int valid = last - (first + i * kTile);
          if (valid < kTile && group == 0) {
            const uint32_t it = 2 * step + 1, slot = it % kSlots;
            ok = mbar_wait_bounded(&ctl.full[slot], (it / kSlots) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            for (int u = valid * 8 + token; u < kTile * 8 && ok; u += 128)
              *reinterpret_cast<uint4*>(smem + Sh::kRing + slot * kTileBytes + u * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          umma::fence_before();
          __syncwarp();
          arrive_if(&ctl.p_full, ok && lane == 0);
        }
      }
      // ----- the columns' results -----------------------------------------------------------
      float l[8], acc[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        umma::unpair(l2[k], l[2 * k], l[2 * k + 1]);
        umma::unpair(acc2[k], acc[2 * k], acc[2 * k + 1]);
      }
      // (sums of 8 columns over 32 lanes: half of the columns change sides at each of three steps)
      float part[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        part[j] = (lane & 16 ? l[j + 4] : l[j]) + __shfl_xor_sync(0xffffffffu, lane & 16 ? l[j] : l[j + 4], 16);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        part[j] = (lane & 8 ? part[j + 2] : part[j]) + __shfl_xor_sync(0xffffffffu, lane & 8 ? part[j] : part[j + 2], 8);
      part[0] = (lane & 4 ? part[1] : part[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? part[0] : part[1], 4);
      part[0] += __shfl_xor_sync(0xffffffffu, part[0], 2);
      part[0] += __shfl_xor_sync(0xffffffffu, part[0], 1);
      if ((lane & 3) == 0) ctl.sum[8 * group + (lane >> 2 & 4) + (lane >> 2 & 2) + (lane >> 2 & 1)][w4] = part[0];
      // Little code from here on: it runs once a piece, and the loop has pushed it out of the
      // instruction caches (unrolled over the columns it took 5000 cycles, 1700 of them to fetch).
      float* stage = reinterpret_cast<float*>(smem + Sh::kStage) + group * 8 * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j) stage[j * 128 + token] = acc[j];
      const bool direct = p.pieces == 1;
      const int live_cols = min(8, cols - 8 * group);
      group_barrier<C / 8>(group);
      if (ok && token < live_cols) {  // a thread a column
        const float4 t = *reinterpret_cast<const float4*>(ctl.sum[8 * group + token]);
        const float total = (t.x + t.y) + (t.z + t.w), top = pick(m, token);  // (0, or 1 at least; or NaN)
        const float m_nat = top == kNothing ? -CUDART_INF_F : top * 0.69314718055994530942f;
        const int64_t row = row_of(token);
        ctl.inverse[8 * group + token] = total == 0.f ? 0.f : 1.f / total;
        if (direct) {
          if (prm.lse != nullptr)
            prm.lse[row] = m_nat == -CUDART_INF_F && total == total ? m_nat : m_nat + logf(total);
          if (S > 1) prm.l_out[row * S] = -1.f;  // nothing to combine
        } else {
          prm.m_out[row * S + p.slot] = m_nat;
          prm.l_out[row * S + p.slot] = total;
          // the sum after the last piece's ends the row's list
          if (p.slot == 0 && p.pieces < S) prm.l_out[row * S + p.pieces] = -1.f;
        }
      }
      if (direct) group_barrier<C / 8>(group);  // the inverses
#pragma unroll 1
      for (int j = w4; j < live_cols && ok; j += 4) {  // a warp a column, a lane 4 channels
        const float4 y = *reinterpret_cast<const float4*>(stage + j * 128 + 4 * lane);
        const int64_t row = row_of(j);
        if (direct) {
          const float f = ctl.inverse[8 * group + j];
          static_cast<uint2*>(prm.out)[row * 32 + lane] =
              make_uint2(mma::pack_bf16(y.x * f, y.y * f), mma::pack_bf16(y.z * f, y.w * f));
        } else {
          reinterpret_cast<float4*>(prm.acc_out)[(row * S + p.slot) * 32 + lane] = y;
        }
      }
    }
    if (!ok && lane == 0) give_up();
    umma::fence_before();
  } else if (warp == Sh::kTmaWarp) {
    // ======================= TMA ==========================================================
    umma::registers_down<Sh::kOtherRegs>();
    const int box_shift = min(page_shift, 6), box_rows = 1 << box_shift;
    const int boxes_of_tile = kTile >> box_shift;  // a lane issues one
    const uint64_t policy = l2_evict_first_policy();
    uint32_t it = 0, handed = 0;
    bool ok = true;
    auto hand_over = [&](const Job& w) {
      const uint32_t s = handed % Sh::kJobs;
      bool free = handed < Sh::kJobs || mbar_wait_bounded(&ctl.job_empty[s], (handed / Sh::kJobs - 1) & 1u);
      free = __all_sync(0xffffffffu, free);
      if (!free) return false;
      if (lane == 0) ctl.jobs[s] = w;
      arrive_if(&ctl.job_full[s], lane == 0);
      __syncwarp();
      ++handed;
      return true;
    };
    Piece p;
    Job job;
    while (ok && walk.next(prm, p)) {
      const int live = min(p.q_len - p.tile * prm.tile_queries, prm.tile_queries);
      const int first = p.c0 * kTile, seen = p.n - p.q_len + p.tile * prm.tile_queries + 1;
      const int last = max(first, min(min(p.n, p.c1 * kTile), seen + live - 1));
      job.first = first;
      job.last = last;
      job.seen = seen;
      job.cols = live * G;
      job.b = p.b;
      job.kvh = p.kvh;
      job.slot = p.slot;
      job.pieces = p.pieces;
      job.row0 = (static_cast<int64_t>(p.q_begin) + p.tile * prm.tile_queries) * prm.num_q_heads + p.kvh * G;
      ok = hand_over(job);
      const int chunks = chunks_of(job);
      const int32_t* pt = prm.page_table + static_cast<int64_t>(p.b) * prm.page_table_stride;
      auto page_of = [&](int i) -> int {
        const int pos = first + i * kTile + lane * box_rows;
        return lane < boxes_of_tile && pos < last ? pt[pos >> page_shift] : -1;
      };
      int next = page_of(0);
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
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const uint32_t slot = it % kSlots;
#ifdef PA_TIMESTAMPS
          // failure-detection test of the instrumented build: after three tiles nothing is issued,
          // so the other warps' waits give up with products in flight
          if (prm.hold_loads && it >= 3) continue;
#endif
          ok = it < kSlots || mbar_wait_bounded(&ctl.empty[slot], (it / kSlots - 1) & 1u);
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
          if (!ok) break;
          if (lane == 0) {
            ctl.issued = static_cast<int>(it) + 1;
            mbar_arrive_expect_tx(&ctl.full[slot], boxes * box_rows * 128);
          }
          __syncwarp();
          if (mine)
            mma::tma_load_4d(base_addr + Sh::kRing + slot * kTileBytes + lane * box_rows * 128,
                             kv ? &map_v : &map_k, 0, pos & (P - 1), p.kvh, page, &ctl.full[slot], policy);
          __syncwarp();
        }
      }
    }
    job.cols = 0;
    ok = hand_over(job) && ok;
    if (!ok && lane == 0) give_up();
  } else if (warp == Sh::kScoreWarp) {
    // ======================= K Q^T ========================================================
    umma::registers_down<Sh::kOtherRegs>();
    if (umma::elect()) {
      constexpr uint32_t kDesc = instruction(Sh::kScoreCols, false);
      const uint32_t q = umma::operand(base_addr + Sh::kQ, 16);
      uint32_t step = 0, piece = 0;
      bool ok = true;
      Job p;
      while (ok && (ok = take(p, true)) && p.cols > 0) {
        const int chunks = chunks_of(p);
        if (chunks == 0) continue;
        ok = mbar_wait_bounded(&ctl.q_full, piece & 1u);
        ++piece;
        for (int i = 0; i < chunks && ok; ++i, ++step) {
          const uint32_t it = 2 * step, slot = it % kSlots, buf = step & 1u;
          ok = mbar_wait_bounded(&ctl.full[slot], (it / kSlots) & 1u);
          if (ok && step >= 2) ok = mbar_wait_bounded(&ctl.s_empty[buf], ((step >> 1) - 1) & 1u);
          if (!ok) break;
          umma::fence_after();
          const uint32_t k = umma::operand(base_addr + Sh::kRing + slot * kTileBytes, 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) 
            mma(tmem + buf * Sh::kScoreCols, k + 2 * j, q + 2 * j, umma::kOperandHigh, kDesc, j > 0);
          umma::commit(&ctl.empty[slot]);
          umma::commit(&ctl.s_full[buf]);
        }
      }
      if (!ok) {
        give_up();
        umma::commit(&ctl.drained[0]);  // what was issued must be over before the memory is freed
        mbar_wait_bounded(&ctl.drained[0], 0);
      }
    }
    __syncwarp();
  } else if (warp == Sh::kOutWarp) {
    // ======================= V^T P^T ======================================================
    umma::registers_down<Sh::kOtherRegs>();
    if (umma::elect()) {
      constexpr uint32_t kDesc = instruction(Sh::kOutCols, true);
      const uint32_t weights = umma::operand(base_addr + Sh::kP, 16);
      uint32_t step = 0;
      bool ok = true;
      Job p;
      while (ok && (ok = take(p, true)) && p.cols > 0) {
        const int chunks = chunks_of(p);
        for (int i = 0; i < chunks && ok; ++i, ++step) {
          const uint32_t it = 2 * step + 1, slot = it % kSlots;
          ok = mbar_wait_bounded(&ctl.full[slot], (it / kSlots) & 1u);
          if (ok) ok = mbar_wait_bounded(&ctl.p_full, step & 1u);
          if (!ok) break;
          umma::fence_after();
          // 32 tokens a step: rows of V, rows of weights
          const uint32_t v = umma::operand(base_addr + Sh::kRing + slot * kTileBytes, 16);
#pragma unroll
          for (int j = 0; j < 4 * Sh::kPasses; ++j) {
            const int pass = j / 4, k = j % 4;
            mma(out_col, v + k * (4096 >> 4), weights + ((pass * Sh::kWeightsTile + k * 32 * Sh::kRowBytes) >> 4),
                Sh::kWeightsHigh, kDesc, j > 0);
          }
          umma::commit(&ctl.empty[slot]);
          umma::commit(&ctl.o_full);
        }
      }
      if (!ok) {
        give_up();
        umma::commit(&ctl.drained[1]);
        mbar_wait_bounded(&ctl.drained[1], 0);
      }
    }
    __syncwarp();
  } else {
    // ======================= the scales ===================================================
    umma::registers_down<Sh::kOtherRegs>();
    // lanes 0 .. 15 have the K scales of up to eight blocks of a chunk, the others V's; a lane's page is asked
    // for two chunks ahead, its scale one
    const int blocks = P >> prm.block_shift, block = lane & 15;
    const bool is_v = lane >= 16, mine = block < kTile >> prm.block_shift;
    const float* scales = is_v ? prm.v_scale : prm.k_scale;
    uint32_t step = 0;
    bool ok = true;
    Job p;
    while (ok && (ok = take(p, false)) && p.cols > 0) {
      const int first = p.first, last = p.last;
      const int chunks = chunks_of(p);
      const int32_t* pt = prm.page_table + static_cast<int64_t>(p.b) * prm.page_table_stride;
      auto pos_of = [&](int i) { return first + i * kTile + (block << prm.block_shift); };
      auto page_of = [&](int i) -> int { return mine && pos_of(i) < last ? pt[pos_of(i) >> page_shift] : 0; };
      auto scale_of = [&](int i, int page) -> float {
        if (!mine || pos_of(i) >= last) return 0.f;
        if (page < 0 || page >= prm.num_pages) page = 0;  // (the TMA warp reports it)
        return scales[(static_cast<int64_t>(page) * prm.num_kv_heads + p.kvh) * blocks +
                      ((pos_of(i) & (P - 1)) >> prm.block_shift)];
      };
      float next = scale_of(0, page_of(0));
      int page = page_of(1);
      for (int i = 0; i < chunks && ok; ++i, ++step) {
        const uint32_t buf = step & 1u;
        const float scale = next;
        next = scale_of(i + 1, page);
        page = page_of(i + 2);
        if (step >= 2) ok = mbar_wait_bounded(&ctl.s_empty[buf], ((step >> 1) - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float v_top = warp_peak(is_v ? fabsf(scale) : 0.f);
        // (a power of two and what undoes it, both normal)
        const int e = max(-126, min(126, 14 - mma::float_exponent(v_top)));
        const float up = v_top < CUDART_INF_F ? __int_as_float((e + 127) << 23) : CUDART_NAN_F;
        if (mine) reinterpret_cast<float*>(&ctl.scales[buf][block])[is_v] = is_v ? scale * up : scale;
        if (lane == 0) ctl.v_down[buf] = __int_as_float((127 - e) << 23);
        __syncwarp();
        arrive_if(&ctl.s_full[buf], lane == 0);
      }
    }
    if (!ok && lane == 0) give_up();
  }
  // (not earlier: with the next launches' blocks waiting beside them these took 137 us, not 95)
  trigger_dependents();
  umma::fence_before();
  __syncthreads();  // every load from tensor memory is over
  if (*abort_flag && tid == 0) {
    // copies in flight must land before the block's memory is given up
    const int issued = *static_cast<volatile int*>(&ctl.issued);
    for (int i = max(0, issued - kSlots); i < issued; ++i)
      mbar_wait_bounded(&ctl.full[i % kSlots], static_cast<uint32_t>(i / kSlots) & 1u);
  }
  if (warp == Sh::kScoreWarp) {
    umma::fence_after();
    dealloc<Sh::kTmemCols>(tmem);
  }
}

// ---- host side ------------------------------------------------------------------------------

template <int C>
cudaError_t launch_one(const BlockParams& p, cudaStream_t stream, bool use_pdl) {
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
  const int64_t most = static_cast<int64_t>(p.sm_count) * Shape<C>::kBlocks;
  const unsigned blocks = static_cast<unsigned>(p.line < most ? p.line : most);
  return fail_at(launch_kernel(block_kernel<C>, dim3(blocks), dim3(Shape<C>::kThreads),
                               static_cast<size_t>(Shape<C>::kBytes), stream, use_pdl, mk, mv, p),
                 "cudaLaunchKernelEx");
}

}  // namespace block
}  // namespace pa

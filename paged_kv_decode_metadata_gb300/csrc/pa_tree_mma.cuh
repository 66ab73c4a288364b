// Tree attention on the 5th-generation tensor cores (tcgen05).
//
// Mathematics.  The G heads of a kv head and the q_len drafted tokens of a request are
// q_len * G rows over the same keys: per kv head S = Q K^T and O += P V are dense products of
// M = 128 rows, 128 tokens and 128 channels.  Softmax is one pass over the tokens: a row's
// weights are 2^(x - r) for a reference r that moves only when a score passes it by more
// than 2^8, so the accumulator is rescaled a few times per split, not per chunk.  Weights
// enter P V rounded to bf16 (2^-8 of each weight's share); their sum l stays unrounded fp32.
// That rounding is chosen for time: what it leaves of a weight as a second bf16 operand brought
// the error against 64 bits from 0.0022-0.0024 to 0.0017, the output's own rounding, and cost
// half as many products again: one request of 1K 12.5 against 11.7 us, 32 of 8K 183 against 169,
// 64 ragged int8 ones 654 against 546, 16 of 16K with 64 drafted 551 against 388.
//
// Shape.  A unit of work is up to 256 rows (two tiles of 128) of one (request, kv head), so a
// K/V chunk of 128 tokens is fetched once for both tiles.  The batch's units are laid end to
// end and cut into equal shares of chunks, one persistent block per SM: ragged batches and
// unit counts that are no multiple of the SMs leave no block idle, and only the units that a
// cut falls into need partials (the rest write their output directly).
// Two streams, each with a score buffer and an accumulator in tensor memory (4 x 128 columns
// = all 512): with two tiles a stream is a tile; with one, the streams take alternate chunks
// and are joined at the end.  So the tensor cores work on one stream while the other's
// softmax runs.
//   warps 0-3, 4-7   softmax of stream 0, 1: a thread owns a row, so maxima and sums need no
//                    exchange; scores come from and weights go back to tensor memory (P
//                    takes the place of S, as the A operand of P V)
//   warp 8           TMA: a ring of four or five 32 KiB tiles, K and V in turn, running ahead
//                    into the next unit; a lane issues one box (up to 64 tokens of one page,
//                    64 channels), so small pages cost no more time than large ones
//   warp 9           issues every MMA: P V of chunk c, then Q K^T of the stream's next chunk,
//                    whose scores are ready when the other stream's are used up
//   warp 10          zeroes V rows past a request's last token (0 * NaN is NaN)
//   warps 12-19      int8 pools: codes to bf16 (exact), from a ring of raw tiles into the ring;
//                    the K scale multiplies the fp32 score, the V scale the weight before
//                    it is rounded
// Masks cost nothing before the last chunks: only chunks that reach the drafted positions
// look at the ancestor bits.
//
// Bound by, bf16: memory up to about 256 rows per kv head (64 KiB of K/V per 128 tokens against
// 1024 tensor cycles per tile), the tensor cores above.  int8: a chunk takes 1.9 us with one
// tile and 2.5 with two (bf16: 1.5 and 1.7).  Widening is four steps a pair of codes on the
// softmax's schedulers, and the widened tiles, the scales and scores in halves (Q read twice)
// keep shared memory about three quarters busy.  Shares weighted by the tiles of a chunk were
// measured and were slower (689 and 731 us against 633 at the time).
// Measured, both launches where a row is cut (heads / kv heads): one request of 1K tokens with 8
// drafted (32 / 8) 11.4 us; 32 requests of 8K with 32 drafted (32 / 8) 168-171 us (6.4 TB/s); 16
// of 16K with 64 drafted (64 / 8) 378-440 us (1.2-1.4 PFLOP/s, under the power cap); 64 ragged
// to 16K, int8, with 32 drafted (64 / 8) 548 us.
#pragma once

#include "pa_splitk_mma.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace tree {

constexpr int kTile = 128;            // rows of a tile, tokens of a chunk
constexpr int kSoftmaxThreads = 256;  // two groups of four warps
constexpr int kTmaWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kConvertWarp = 12, kConvertWarps = 8;
// Threads of a block.  The softmax warps (a row's 128 scores in registers, int8: 64 at a time)
// and the others split the registers that the block was launched with.  int8: eight widening
// warps, not four: 1.88 against 2.19 us a chunk with one tile, as fast with two.
template <bool kQuant>
struct Roles {
  static constexpr int kThreads = kQuant ? 640 : 384;
  static constexpr int kLaunchRegs = kQuant ? 96 : 168;  // what fits the threads into 65,536
  static constexpr int kSoftmaxRegs = kQuant ? 128 : 216, kOtherRegs = 72;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs,
                "register split");
};
constexpr int kHalfBytes = kTile * 128;       // 64 channels of 128 rows
constexpr int kTileBytes = 2 * kHalfBytes;
// int8: codes of a tile as they come, and behind a K tile's the chunk's K and V scales
constexpr int kRawCodes = kTile * 128;
constexpr int kRawBytes = kRawCodes + 2 * kTile * 4;
constexpr int kScaleSlots = 4;

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

// One piece of work: chunks [c0, c1) of one unit.  A unit is up to 256 rows (two tiles) of a
// (request, kv head); the units of a request follow one another kv head by kv head.
struct Piece {
  int b, q_begin, q_len, n;  // the request, its query rows, its cached tokens
  int kvh, pair;
  int c0, c1;
  int slot, pieces;  // which of the unit's pieces this is, and how many it has
};

// The batch as one line of chunks, unit after unit, cut into equal shares: block i takes
// [i share, (i + 1) share), or several shares in a row where one each would be longer than a
// piece should be.  Every warp walks its block's shares by itself.  (The host keeps the
// line's length within 31 bits.)
struct Walk {
  int b, q_begin, q_len, n, pairs, chunks;  // the request at hand
  int base, pos, end, share;                // its start on the line; where the walk is
  int at_share;                             // and in which share; -1: units are not cut

  // Lengths of request r, checked; `report` records what is wrong with them.  False: its query
  // rows are refused.
  __device__ __forceinline__ bool load(const TreeParams& prm, int page_size, int r, bool report) {
    b = r;
    q_begin = prm.cu_seqlens_q[r];
    q_len = prm.cu_seqlens_q[r + 1] - q_begin;
    n = prm.cache_seqlens[r];
    const bool fits =
        q_begin >= 0 && q_len >= 0 && q_len <= prm.max_q_len && q_begin <= prm.total_q - q_len;
    if (!fits) {
      if (report) record_error(prm.err, kErrSeqLenOutOfRange);
      q_len = 0;
    }
    const int cap = prm.max_seq_pages * page_size;
    if (n < 0 || n > cap) {
      if (report) record_error(prm.err, kErrSeqLenOutOfRange);
      n = n < 0 ? 0 : cap;
    }
    pairs = ((q_len << prm.group_shift) + 2 * kTile - 1) / (2 * kTile);
    chunks = (n + kTile - 1) / kTile;
    return fits;
  }
  __device__ __forceinline__ int length(const TreeParams& prm) const {
    return pairs * prm.num_kv_heads * chunks;
  }

  // Whole-warp: finds the block's share.  Returns kEmpties where some request has queries but
  // nothing cached (its rows are no work, but have a result), kGaps where rows before the last
  // request's end belong to none: those before the first request's and refused ones.
  static constexpr uint32_t kEmpties = 1, kGaps = 2;
  __device__ __forceinline__ uint32_t start(const TreeParams& prm, int page_size, int lane, bool report) {
    int total = 0, first_sum = 0, first_w = 0;  // the first 32 requests' lengths are kept
    int longest = 0, shortest = INT_MAX;        // units, in chunks
    uint32_t special = 0;
    for (int r0 = 0; r0 < prm.bs; r0 += 32) {
      int w = 0;
      if (r0 + lane < prm.bs) {
        const bool fits = load(prm, page_size, r0 + lane, report);
        w = length(prm);
        if (!fits || (r0 + lane == 0 && q_begin != 0)) special |= kGaps;
        if (q_len > 0 && n == 0) special |= kEmpties;
        if (w > 0) {
          longest = max(longest, chunks);
          shortest = min(shortest, chunks);
        }
      }
      int incl = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      if (r0 == 0) {
        first_sum = incl;
        first_w = w;
      }
      total += __shfl_sync(0xffffffffu, incl, 31);
    }
    special = __reduce_or_sync(0xffffffffu, special);
    const int grid = static_cast<int>(gridDim.x);
    longest = __reduce_max_sync(0xffffffffu, longest);
    shortest = __reduce_min_sync(0xffffffffu, shortest);
    const int even = (total + grid - 1) / grid;
    // A unit of c chunks meets at most floor((c - 1) / share) + 2 shares (c of them if share is
    // 1): a share of longest / (num_splits - 1) keeps every unit's pieces within num_splits.
    // (From the lengths, not from the page table's width: under a table for 1M tokens that left
    // most SMs without work, 8 requests of 8K taking 1550 us against 54.)
    const int S = prm.num_splits;
    int rounds = max(1, (even + kTreePieceChunks - 1) / kTreePieceChunks);  // shares per block
    share = (even + rounds - 1) / rounds;
    if (S > 1 && S < longest) share = max(share, (longest + S - 2) / (S - 1));
    if (rounds > 1) rounds = (even + share - 1) / share;
    // Units of one length that fill the blocks well enough stay whole: partials and their
    // join cost more than up to a quarter of a share left idle (256 units on 152 SMs: whole
    // 169 / 382 us, cut 179 / 407 us for one and two tiles).
    const bool whole =
        S == 1 || (longest == shortest && longest <= kTreePieceChunks &&
                   (total / longest + grid - 1) / grid * longest <= rounds * share + rounds * share / 4);
    const int own = whole ? even : rounds * share;  // of the line, this block's
    const long long at_ll = static_cast<long long>(blockIdx.x) * own;
    pos = static_cast<int>(min(at_ll, static_cast<long long>(total)));
    at_share = whole ? -1 : static_cast<int>(blockIdx.x) * rounds;
    end = static_cast<int>(min(at_ll + own, static_cast<long long>(total)));
    if (pos >= end) return special;
    // the request that holds pos and, where units are not cut, the unit starts at or after
    // pos and end
    int at = 0, new_end = end < total ? end : total, found = -1, found_base = 0;
    bool end_found = !whole || end == total;
    for (int r0 = 0; r0 < prm.bs && !(found >= 0 && end_found); r0 += 32) {
      int w = first_w, incl = first_sum;
      if (r0 > 0) {
        w = 0;
        if (r0 + lane < prm.bs) {
          load(prm, page_size, r0 + lane, false);
          w = length(prm);
        }
        incl = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += up;
        }
      }
      const int first = at + incl - w;
      const uint32_t has = __ballot_sync(0xffffffffu, first <= pos && pos < first + w);
      if (has != 0) {
        found = r0 + __ffs(has) - 1;
        found_base = __shfl_sync(0xffffffffu, first, __ffs(has) - 1);
      }
      const uint32_t last = __ballot_sync(0xffffffffu, first <= end && end < first + w);
      if (whole && last != 0) {
        load(prm, page_size, r0 + __ffs(last) - 1, false);
        const int f = __shfl_sync(0xffffffffu, first, __ffs(last) - 1);
        new_end = f + (end - f + chunks - 1) / chunks * chunks;
        end_found = true;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (prm.bs <= 32 && !whole) {  // the lane that holds it has its lengths
      b = found;
      q_begin = __shfl_sync(0xffffffffu, q_begin, found);
      q_len = __shfl_sync(0xffffffffu, q_len, found);
      n = __shfl_sync(0xffffffffu, n, found);
      pairs = __shfl_sync(0xffffffffu, pairs, found);
      chunks = __shfl_sync(0xffffffffu, chunks, found);
    } else {
      load(prm, page_size, found, false);  // (found >= 0: pos lies on the line)
    }
    base = found_base;
    if (whole) {
      pos = base + (pos - base + chunks - 1) / chunks * chunks;
      end = new_end;
    }
    return special;
  }

  __device__ __forceinline__ bool next(const TreeParams& prm, int page_size, Piece& p) {
    if (pos >= end) return false;
    while (pos - base >= length(prm)) {  // into the next request that has work
      base += length(prm);
      load(prm, page_size, b + 1, false);
    }
    const int unit = (pos - base) / chunks, from = base + unit * chunks;
    p.b = b;
    p.q_begin = q_begin;
    p.q_len = q_len;
    p.n = n;
    p.kvh = unit / pairs;
    p.pair = unit - p.kvh * pairs;
    p.c0 = pos - from;
    p.c1 = min(chunks, end - from);
    p.slot = 0;
    p.pieces = 1;
    if (at_share >= 0) {
      const int first = from / share, edge = (at_share + 1) * share;
      p.c1 = min(p.c1, edge - from);
      p.slot = at_share - first;
      at_share += from + p.c1 == edge;
      p.pieces = (from + chunks - 1) / share - first + 1;
    }
    pos = from + p.c1;
    return true;
  }
};

// Shared memory of a block: the Q tiles, the ring, the softmax warps' way out, the control
// words.  kTiles: Q tiles of the batch's units; with one, the other's room is a ring tile
// more (memory bound there: two V tiles are held by the streams, the rest is in flight).
// int8: the ring holds the widened tiles, three (so that widening V of a chunk does not wait for
// the products of the chunk before) or, with one Q tile, four (nor K of the chunk after next
// for this one's); the raw tiles behind it are what is in flight.
template <int kTiles, bool kQuant>
struct Shared {
  static constexpr int kSlots = kQuant ? 5 - kTiles : 6 - kTiles;
  static constexpr int kRawSlots = 2;  // (a third: no faster)
  static constexpr int kLinePieces = kQuant ? 4 : 8;  // 16-byte pieces of a row on the way out
  static constexpr int kStageBytes = 32 * 16 * kLinePieces;  // per softmax warp
  static constexpr int kQ = 0;
  static constexpr int kRing = kTiles * kTileBytes;
  static constexpr int kRaw = kRing + kSlots * kTileBytes;
  static constexpr int kScales = kRaw + (kQuant ? kRawSlots * kRawBytes : 0);
  static constexpr int kStage = kScales + (kQuant ? kScaleSlots * 2 * kTile * 4 : 0);
  static constexpr int kEnd = kStage + kSoftmaxThreads / 32 * kStageBytes;
  struct Control {
    uint64_t full[kSlots], empty[kSlots], raw_full[kRawSlots], raw_empty[kRawSlots];
    uint64_t q_full, q_empty, o_full[2], drained;
    // by ring tile: a request's last V tile on its way to the cleaning warp.  (One for all would
    // not do: the next short request's tile may be issued before this one has landed.)
    uint64_t v_last[kSlots];
    // bf16: a stream's scores, the first half of its weights, all of them; int8: [stream][half
    // of the chunk], and each product's end
    uint64_t s_full[4], p_half[2], p_ready[4], pv_done[2];
    Walk walk[kSoftmaxThreads / 32];  // of the softmax warps
    Piece piece[kSoftmaxThreads / 32];
    float join[2][kTile];  // one number a row, from stream to stream
    uint32_t tmem;
    int abort, issued, issued_q;
    int issued_v[kSlots];
  };
  static constexpr int kBytes = kEnd + static_cast<int>(sizeof(Control)) + 1024;  // + alignment
  static_assert(kBytes <= 227 * 1024, "one block's shared memory");
};

// Four int8 codes -> two words of two bf16 each, exactly.  A byte b = 128 s + m (s the sign
// bit, m the low seven) behind 0x43 reads as 128 + m with the sign bit cleared and as 128 (1 +
// s) with m cleared; the difference is m - 128 s, the code.
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t word, uint32_t selector) {
  const uint32_t t = __byte_perm(word, 0x43434343u, selector);
  const uint32_t x = t & 0xff7fff7fu, y = t & 0xff80ff80u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&d);
}

template <int P, int kTiles, bool kQuant>
__global__ void __launch_bounds__(Roles<kQuant>::kThreads, 1)
    tree_mma_kernel(const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const TreeParams prm) {
  using Sh = Shared<kTiles, kQuant>;
  using Ro = Roles<kQuant>;
  constexpr int kThreads = Ro::kThreads;
  constexpr int kSlots = Sh::kSlots, kRawSlots = Sh::kRawSlots;
  extern __shared__ unsigned char smem_raw[];
  // (rounded up by an offset, not by way of an integer: the compiler then still knows that it
  // is shared memory, and the generic accesses it would use otherwise took four times as long)
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const uint32_t base_addr = smem_addr(smem);
  typename Sh::Control& ctl = *reinterpret_cast<typename Sh::Control*>(smem + Sh::kEnd);
  volatile int* abort_flag = &ctl.abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform for the compiler too)
  const int gs = prm.group_shift, G = 1 << gs;  // heads of a kv head: a power of two
  const int S = prm.num_splits;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.full[i], kQuant ? kConvertWarps : 1);  // int8: the widening warps
      mbar_init(&ctl.empty[i], 1);
      mbar_init(&ctl.v_last[i], 1);
      ctl.issued_v[i] = 0;
    }
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(&ctl.raw_full[i], 1);
      mbar_init(&ctl.raw_empty[i], kConvertWarps);
    }
    mbar_init(&ctl.q_full, 1);
    mbar_init(&ctl.q_empty, 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ctl.s_full[s], 1);
      mbar_init(&ctl.p_ready[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.p_half[s], 4);
      mbar_init(&ctl.o_full[s], 1);
      mbar_init(&ctl.pv_done[s], 1);
    }
    mbar_init(&ctl.drained, 1);
    ctl.abort = 0;
    ctl.issued = 0;
    ctl.issued_q = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) umma::alloc_all(&ctl.tmem);
  grid_dependency_wait();

  Walk walk;
  const uint32_t special = walk.start(prm, P, lane, blockIdx.x == 0 && warp == 0);
  if (special & Walk::kEmpties) {  // requests with queries and an empty cache
    Walk w;
    for (int r = blockIdx.x; r < prm.bs; r += gridDim.x) {
      w.load(prm, P, r, false);
      if (w.n > 0) continue;
      const int64_t first = static_cast<int64_t>(w.q_begin) * prm.num_q_heads;
      for (int i = tid; i < w.q_len * prm.num_q_heads; i += kThreads) {
        if (prm.lse != nullptr) prm.lse[first + i] = -CUDART_INF_F;
        if (S > 1) prm.l_out[(first + i) * S] = -1.f;
      }
      for (int i = tid; i < w.q_len * prm.num_q_heads * 16; i += kThreads)
        static_cast<uint4*>(prm.out)[first * 16 + i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if ((special & Walk::kGaps) && S > 1) {  // the join leaves a row alone whose first sum is negative
    const int rows = max(0, min(prm.cu_seqlens_q[prm.bs], prm.total_q));
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kThreads + tid; row < rows;
         row += static_cast<int64_t>(gridDim.x) * kThreads) {
      Walk w;
      bool covered = false;
      for (int r = 0; r < prm.bs && !covered; ++r) {
        w.load(prm, P, r, false);
        covered = row >= w.q_begin && row < w.q_begin + w.q_len;
      }
      for (int h = 0; h < prm.num_q_heads && !covered; ++h)
        prm.l_out[(row * prm.num_q_heads + h) * S] = -1.f;
    }
  }

  if (warp < kTmaWarp && lane == 0) ctl.walk[warp] = walk;
  umma::fence_before();
  __syncthreads();  // barriers initialised, tensor memory allocated
  umma::fence_after();
  const uint32_t tmem = ctl.tmem;
  // columns: scores (and weights) of stream s at 128 s, accumulator at 256 + 128 s
  auto s_col = [&](int s) { return tmem + static_cast<uint32_t>(s) * kTile; };
  auto o_col = [&](int s) { return tmem + 256u + static_cast<uint32_t>(s) * kTile; };
  auto give_up = [&]() {
    record_error(prm.err, kErrWaitTimeout);
    *abort_flag = 1;
  };
  // two tiles: each is a stream over every chunk; one: the streams take alternate chunks
  auto two_tiles = [&](const Piece& p) {
    return kTiles == 2 && p.q_len * G - p.pair * 2 * kTile > kTile;
  };
  auto stream_chunks = [](bool two, int chunks, int s) { return two ? chunks : (chunks + 1 - s) / 2; };

  if (warp < kTmaWarp) {
    // ======================= softmax ===================================================
    umma::registers_up<Ro::kSoftmaxRegs>();
    const int s = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 (warp % 4)
    const uint32_t sc = s_col(s) + lane_base, oc = o_col(s) + lane_base;
    const float scale = prm.q_scale;
    const int words = 2 * prm.mask_words;
    uint32_t step = 0, outputs = 0;  // of this stream, over all pieces
    uint32_t chunk0 = 0;             // chunks of the pieces before
    // (after a wait that gave up, the pieces that are left only meet the barriers of the
    // softmax warps, so that none of them waits there for good)
    bool ok = true;
    // A thread's registers hold a row of scores, so the walk and the piece stay in shared
    // memory: `volatile` has them read again where they are needed.
    const volatile Piece& vp = ctl.piece[warp];
    while (true) {
      __syncwarp();
      if (lane == 0) {
        Walk w = ctl.walk[warp];
        Piece next;
        next.c1 = 0;
        w.next(prm, P, next);
        ctl.walk[warp] = w;
        ctl.piece[warp] = next;
      }
      __syncwarp();
      if (vp.c1 == 0) break;
      const bool two = kTiles == 2 && vp.q_len * G - vp.pair * 2 * kTile > kTile;
      // this stream's chunks: c0 + k (two tiles) or c0 + 2 k + s; from `plain` on they reach the
      // drafted positions
      const int mine = stream_chunks(two, vp.c1 - vp.c0, s);
      const int committed = max(0, vp.n - vp.q_len) / kTile - vp.c0;  // chunks of those alone
      const int plain = two ? committed : (committed - s + 1) >> 1;
      float m_ref = -CUDART_INF_F, l = 0.f;  // the row's reference and sum of weights
      for (int k = 0; k < mine && ok; ++k) {
        if constexpr (kQuant) {
          // Half a chunk at a time, each half with its own scores in tensor memory: while one
          // half's weights are made, the tensor cores work on the other's.
          const float4* scales = reinterpret_cast<const float4*>(smem + Sh::kScales) +
                                 (chunk0 + (two ? k : 2 * k + s)) % kScaleSlots * (2 * kTile / 4);
          // (the chunk's K scales times the softmax scale, then its V scales; written before the
          // scores' K tile was handed on, so before these scores)
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            ok = mbar_wait_bounded(&ctl.s_full[2 * s + half], step & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            umma::fence_after();
            const uint32_t at = sc + 64 * half;
            const float4* f_of = scales + 16 * half;
            float x[64];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              umma::ld32(at + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * i]));
#pragma unroll
            for (int i = 0; i < 2; ++i) umma::wait_ld(*reinterpret_cast<uint32_t(*)[32]>(&x[32 * i]));
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
              const float4 f = f_of[j / 4];
              umma::unpair(umma::mul2(umma::pair(x[j], x[j + 1]), umma::pair(f.x, f.y)), x[j], x[j + 1]);
              umma::unpair(umma::mul2(umma::pair(x[j + 2], x[j + 3]), umma::pair(f.z, f.w)), x[j + 2],
                           x[j + 3]);
            }
            if (k >= plain) {  // drafted or missing positions
              const int row = (vp.pair * 2 + (two ? s : 0)) * kTile + r;
              const int q_len = vp.q_len, n = vp.n;
              const bool live = row < q_len * G;
              const uint32_t* mask =
                  prm.tree_mask + (static_cast<int64_t>(vp.q_begin) + (live ? row >> gs : 0)) * words;
              const int p0 = (vp.c0 + (two ? k : 2 * k + s)) * kTile + 64 * half;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t bits = live ? visible(p0 + 32 * i, n - q_len, n, mask, words) : 0u;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  x[32 * i + j] = (bits >> j) & 1u ? x[32 * i + j] : -CUDART_INF_F;
              }
              __syncwarp();
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < 60; j += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u) mx[u] = umma::max3(mx[u], x[j + u], x[j + 4 + u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], x[60 + u]);
            const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            float alpha = 1.f;
            if (m_new > m_ref + mma::kMaxSlack) {
              alpha = m_ref == -CUDART_INF_F ? 0.f : mma::fast_exp2(m_ref - m_new);
              m_ref = m_new;
              l *= alpha;
            }
            __syncwarp();
            // The accumulator follows a moved reference, once the last product is over (before
            // the piece's first there is none).
            if (k + half > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
              ok = mbar_wait_bounded(&ctl.pv_done[s], (2 * step + half - 1) & 1u);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              umma::fence_after();
#pragma unroll 1
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
            const uint64_t ref2 = umma::pair(-ref, -ref);
            uint64_t sum[4] = {0, 0, 0, 0};  // pairs of +0
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float4 g4 = f_of[kTile / 4 + 8 * i + j / 2];
                const float2 g = j & 1 ? make_float2(g4.z, g4.w) : make_float2(g4.x, g4.y);
                float lo, hi;
                umma::unpair(umma::add2(umma::pair(x[32 * i + 2 * j], x[32 * i + 2 * j + 1]), ref2), lo, hi);
                lo = mma::fast_exp2(lo);
                hi = mma::fast_exp2(hi);
                sum[j & 3] = umma::add2(sum[j & 3], umma::pair(lo, hi));
                // the V scale goes with the weight
                umma::unpair(umma::mul2(umma::pair(lo, hi), umma::pair(g.x, g.y)), lo, hi);
                w[j] = mma::pack_bf16(lo, hi);
              }
              umma::st16(at + 16 * i, w);
            }
            umma::wait_st();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mma::mbar_arrive(&ctl.p_ready[2 * s + half]);
            float lo, hi;
            umma::unpair(umma::add2(umma::add2(sum[0], sum[1]), umma::add2(sum[2], sum[3])), lo, hi);
            l += lo + hi;
          }
          if (!ok) break;
          ++step;
        } else {
          ok = mbar_wait_bounded(&ctl.s_full[s], step & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++step;
          umma::fence_after();
          float x[kTile];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            umma::ld32(sc + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * i]));
#pragma unroll
          for (int i = 0; i < 4; ++i) umma::wait_ld(*reinterpret_cast<uint32_t(*)[32]>(&x[32 * i]));
          if (k >= plain) {  // drafted or missing positions
            const int row = (vp.pair * 2 + (two ? s : 0)) * kTile + r;
            const int q_len = vp.q_len, n = vp.n;
            const bool live = row < q_len * G;
            const uint32_t* mask =
                prm.tree_mask + (static_cast<int64_t>(vp.q_begin) + (live ? row >> gs : 0)) * words;
            const int p0 = (vp.c0 + (two ? k : 2 * k + s)) * kTile;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t bits = live ? visible(p0 + 32 * i, n - q_len, n, mask, words) : 0u;
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
          // the accumulator follows a moved reference (before the first product there is none;
          // earlier products are over once the scores are)
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
            if (i & 1) {  // half of the weights: their products may start
              umma::wait_st();
              umma::fence_before();
              __syncwarp();
              if (lane == 0) mma::mbar_arrive(i == 1 ? &ctl.p_half[s] : &ctl.p_ready[s]);
            }
          }
          float lo, hi;
          umma::unpair(umma::add2(umma::add2(sum[0], sum[1]), umma::add2(sum[2], sum[3])), lo, hi);
          l += lo + hi;
        }
      }
      chunk0 += vp.c1 - vp.c0;
      // ----- the rows' results -------------------------------------------------------------
      if (ok && mine > 0) {
        ok = mbar_wait_bounded(&ctl.o_full[s], outputs & 1u);
        ok = __all_sync(0xffffffffu, ok);
        ++outputs;
      }
      if (!ok && lane == 0) give_up();
      umma::fence_after();
      const Piece p = {vp.b, vp.q_begin, vp.q_len, vp.n, vp.kvh, vp.pair, vp.c0, vp.c1, vp.slot, vp.pieces};
      const int row = (p.pair * 2 + (two ? s : 0)) * kTile + r;
      const bool live = row < p.q_len * G;
      const int qi = live ? row >> gs : 0;
      const int64_t slot = (static_cast<int64_t>(p.q_begin) + qi) * prm.num_q_heads + p.kvh * G +
                           (live ? row - qi * G : 0);
      float f_own = 1.f, f_other = 0.f;  // factors of this and the other stream's accumulator
      int col0 = 0, col1 = kTile;        // channels this thread writes
      if (!two && p.c1 - p.c0 > 1) {
        // one tile: join the streams (both see each other's accumulator: the same lanes);
        // each writes half of the channels
        float* box = ctl.join[s];
        box[r] = m_ref;
        umma::fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        umma::fence_after();
        const float m_other = ctl.join[1 - s][r];
        asm volatile("bar.sync 1, 256;" ::: "memory");
        box[r] = l;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float m_all = fmaxf(m_ref, m_other);
        f_own = m_ref == -CUDART_INF_F ? 0.f : mma::fast_exp2(m_ref - m_all);
        f_other = m_other == -CUDART_INF_F ? 0.f : mma::fast_exp2(m_other - m_all);
        l = l * f_own + ctl.join[1 - s][r] * f_other;
        m_ref = m_all;
        col0 = s * (kTile / 2);
        col1 = col0 + kTile / 2;
      } else if (!two && s == 1) {
        col1 = 0;  // a single chunk: stream 0 has it all
      }
      const bool direct = p.pieces == 1;
      const float inv = direct ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      const uint32_t other = o_col(1 - s) + lane_base;
      const bool write = live && ok;
      // Rows leave through shared memory, a line (128 bytes, int8: 64) of each of the warp's 32
      // at a time, so that a store covers lines of several rows: storing a row per thread took
      // 32 lines a store and held up every other warp's shared-memory work for 8K cycles.
      // (16-byte pieces are XORed with the row: few bank conflicts either way.)
      constexpr int kLine = Sh::kLinePieces;
      uint4* stage = reinterpret_cast<uint4*>(smem + Sh::kStage + warp * Sh::kStageBytes);
      const int row0 = (p.pair * 2 + (two ? s : 0)) * kTile + (warp & 3) * 32;
      const int live_rows = ok ? p.q_len * G - row0 : 0;  // of the warp's 32
      auto put = [&](int piece, uint4 w) { stage[lane * kLine + (piece ^ (lane & (kLine - 1)))] = w; };
      // the line at 16-byte piece `at` of every row
      auto flush = [&](int at) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLine; ++i) {
          const int rr = (32 / kLine) * i + lane / kLine, piece = lane & (kLine - 1);
          if (rr < live_rows) {
            const uint4 w = stage[rr * kLine + (piece ^ (rr & (kLine - 1)))];
            const int q = (row0 + rr) >> gs;
            const int64_t to = (static_cast<int64_t>(p.q_begin) + q) * prm.num_q_heads + p.kvh * G +
                               (row0 + rr - q * G);
            if (direct) {
              static_cast<uint4*>(prm.out)[to * 16 + at + piece] = w;
            } else {
              reinterpret_cast<uint4*>(prm.acc_out)[(to * S + p.slot) * 32 + at + piece] = w;
            }
          }
        }
        __syncwarp();
      };
      for (int c = col0; c < col1; c += 32) {
        float y[32];
        uint32_t o[32];
        __syncwarp();
        umma::ld32(oc + c, o);
        umma::wait_ld(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(o[j]) * f_own;
        if (!two) {
          umma::ld32(other + c, o);
          umma::wait_ld(o);
          // (without a second chunk the other accumulator holds nothing of this piece)
          if (f_other != 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = fmaf(__uint_as_float(o[j]), f_other, y[j]);
          }
          __syncwarp();
        }
        if (direct) {
          const int first = c / 8 & (kLine - 1);  // bf16: 32 channels are four pieces
#pragma unroll
          for (int j = 0; j < 4; ++j)
            put(first + j, make_uint4(mma::pack_bf16(y[8 * j] * inv, y[8 * j + 1] * inv),
                                      mma::pack_bf16(y[8 * j + 2] * inv, y[8 * j + 3] * inv),
                                      mma::pack_bf16(y[8 * j + 4] * inv, y[8 * j + 5] * inv),
                                      mma::pack_bf16(y[8 * j + 6] * inv, y[8 * j + 7] * inv)));
          if (first + 4 == kLine) flush(c / 8 + 4 - kLine);
        } else {  // fp32: eight pieces
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            put(j & (kLine - 1), make_uint4(__float_as_uint(y[4 * j]), __float_as_uint(y[4 * j + 1]),
                                            __float_as_uint(y[4 * j + 2]), __float_as_uint(y[4 * j + 3])));
            if ((j & (kLine - 1)) == kLine - 1) flush(c / 4 + j + 1 - kLine);
          }
        }
      }
      if (write && (two || s == 0)) {
        const float m_nat = m_ref * 0.69314718055994530942f;  // -inf stays -inf
        if (direct) {
          // (l is NaN where a score was: m_ref, a maximum, does not show it)
          if (prm.lse != nullptr)
            prm.lse[slot] = m_ref == -CUDART_INF_F && l == l ? m_ref : m_nat + logf(l);
          if (S > 1) prm.l_out[slot * S] = -1.f;  // nothing to combine
        } else {
          prm.m_out[slot * S + p.slot] = m_nat;
          prm.l_out[slot * S + p.slot] = l;
          // the sum after the last piece's ends the row's list
          if (p.slot == 0 && p.pieces < S) prm.l_out[slot * S + p.pieces] = -1.f;
        }
      }
      umma::fence_before();
      // neither stream's next product may overwrite an accumulator that the other reads, nor
      // the next join this one's numbers
      if (!two) asm volatile("bar.sync 1, 256;" ::: "memory");
    }
  } else if (kQuant && warp >= kConvertWarp) {
    // ======================= int8: codes to bf16 ============================================
    umma::registers_down<Ro::kOtherRegs>();
    Piece p;
    const int t = tid - kConvertWarp * 32;  // 0..255
    // A warp turns 8 rows x 4 pieces of 16 codes at a time: every row's swizzle puts its piece
    // in another bank group, for the loads and for both stores.  Offsets of the warp's first
    // rows; the other four pieces of a row and the piece's second half are a bit away.
    const int first_row = ((warp - kConvertWarp) * 16 + (lane & 7)) * 128;
    const int from = first_row + (((lane >> 3) ^ (lane & 7)) << 4);
    const int to = first_row + (((2 * (lane >> 3)) ^ (lane & 7)) << 4);
    int it = 0;
    uint32_t chunk = 0;
    bool ok = true;
    while (ok && walk.next(prm, P, p)) {
      for (int c = p.c0; c < p.c1 && ok; ++c, ++chunk) {
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int raw = it % kRawSlots, slot = it % kSlots;
          ok = mbar_wait_bounded(&ctl.raw_full[raw], static_cast<uint32_t>(it / kRawSlots) & 1u) &&
               (it < kSlots ||
                mbar_wait_bounded(&ctl.empty[slot], static_cast<uint32_t>(it / kSlots - 1) & 1u));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const unsigned char* src = smem + Sh::kRaw + raw * kRawBytes;
          unsigned char* dst = smem + Sh::kRing + slot * kTileBytes;
          if (kv == 0) {
            // V scales of positions past the end may hold anything, and 0 * NaN is NaN
            const float* in = reinterpret_cast<const float*>(src + kRawCodes);
            float* out = reinterpret_cast<float*>(smem + Sh::kScales) + chunk % kScaleSlots * 2 * kTile;
            out[t] = t < kTile ? in[t] * prm.q_scale : (c - 1) * kTile + t < p.n ? in[t] : 0.f;
          }
          // four pieces are loaded before the first store: the compiler cannot know that the two
          // tiles do not overlap
          {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = *reinterpret_cast<const uint4*>(src + (u >> 1) * 1024 + (u & 1 ? from ^ 64 : from));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              unsigned char* half = dst + (u >> 1) * 1024 + (u & 1) * kHalfBytes;
              *reinterpret_cast<uint4*>(half + to) =
                  make_uint4(codes_to_bf16x2(w[u].x, 0x4140), codes_to_bf16x2(w[u].x, 0x4342),
                             codes_to_bf16x2(w[u].y, 0x4140), codes_to_bf16x2(w[u].y, 0x4342));
              *reinterpret_cast<uint4*>(half + (to ^ 16)) =
                  make_uint4(codes_to_bf16x2(w[u].z, 0x4140), codes_to_bf16x2(w[u].z, 0x4342),
                             codes_to_bf16x2(w[u].w, 0x4140), codes_to_bf16x2(w[u].w, 0x4342));
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mma::mbar_arrive(&ctl.full[slot]);
            mma::mbar_arrive(&ctl.raw_empty[raw]);
          }
        }
      }
    }
    if (!ok && lane == 0) give_up();
  } else {
    umma::registers_down<Ro::kOtherRegs>();
    Piece p;
    if (warp == kTmaWarp) {
      // ======================= TMA ======================================================
      constexpr int kBoxRows = P < 64 ? P : 64;
      constexpr int kBoxes = kTile / kBoxRows;
      const uint64_t policy = l2_evict_first_policy();
      // lane -> (box of the chunk, channel half)
      // (int8: lane -> box and what of it: the codes, and with K its K and its V scales)
      const int box = kQuant ? lane & 7 : lane >> 1, half = kQuant ? lane >> 3 : lane & 1;
      int it = 0;  // ring tiles issued
      uint32_t piece = 0;
      bool ok = true, more = walk.next(prm, P, p);
      auto load_rows = [&]() {  // Q of piece p; lane 0
        const int tiles = two_tiles(p) ? 2 : 1;
        ctl.issued_q = piece + 1;
        mbar_arrive_expect_tx(&ctl.q_full, tiles * kTileBytes);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < 2; ++h)
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(base_addr + Sh::kQ + t * kTileBytes +
                                                       h * kHalfBytes),
                "l"(reinterpret_cast<uint64_t>(&map_q)), "r"(64 * h), "r"(p.kvh * G),
                "r"(p.q_begin + (p.pair * 2 + t) * (kTile >> gs)), "r"(smem_addr(&ctl.q_full))
                : "memory");
      };
      if (more && lane == 0) load_rows();
      __syncwarp();
      while (ok && more) {
        const int32_t* pt = prm.page_table + static_cast<int64_t>(p.b) * prm.page_table_stride;
        auto token_of = [&](int c) { return c * kTile + box * kBoxRows; };
        auto page_of = [&](int c) -> int {  // this lane's page of chunk c, -1: nothing to load
          const int tok = token_of(c);
          return c < p.c1 && box < kBoxes && tok < p.n ? pt[tok / P] : -1;
        };
        int next = page_of(p.c0);
        for (int c = p.c0; c < p.c1 && ok; ++c) {
          const int tok = token_of(c);
          const bool mine = box < kBoxes && tok < p.n;
          int pg = next;
          next = page_of(c + 1);
          if (mine && (pg < 0 || pg >= prm.num_pages)) {
            record_error(prm.err, kErrPageOutOfRange);
            pg = 0;
          }
          const int boxes = min(kBoxes, (p.n - c * kTile + kBoxRows - 1) / kBoxRows);
          for (int kv = 0; kv < 2; ++kv, ++it) {
#ifdef PA_TIMESTAMPS
            // failure-detection test of the instrumented build: after three tiles nothing is
            // issued, so the other warps' waits give up with products in flight
            if (prm.hold_loads && it >= 3) break;
#endif
            if constexpr (kQuant) {
              const int slot = it % kRawSlots;
              ok = it < kRawSlots || mbar_wait_bounded(&ctl.raw_empty[slot],
                                                       static_cast<uint32_t>(it / kRawSlots - 1) & 1u);
              ok = __all_sync(0xffffffffu, ok && !*abort_flag);
              if (!ok) break;
              if (lane == 0) {
                ctl.issued = it + 1;
                mbar_arrive_expect_tx(&ctl.raw_full[slot],
                                      boxes * kBoxRows * (128 + (kv == 0 ? 2 * 4 : 0)));
              }
              __syncwarp();
              const uint32_t at = base_addr + Sh::kRaw + slot * kRawBytes;
              if (mine && half == 0) {
                mma::tma_load_4d(at + box * kBoxRows * 128, kv ? &map_v : &map_k, 0, tok % P, p.kvh, pg,
                                 &ctl.raw_full[slot], policy);
              } else if (mine && half <= 2 && kv == 0) {
                const int64_t row = (static_cast<int64_t>(pg) * prm.num_kv_heads + p.kvh) * P + tok % P;
                bulk_copy_g2s(smem + Sh::kRaw + slot * kRawBytes + kRawCodes +
                                  ((half - 1) * kTile + box * kBoxRows) * 4,
                              (half == 1 ? prm.k_scale : prm.v_scale) + row, kBoxRows * 4,
                              &ctl.raw_full[slot], policy);
              }
              __syncwarp();
              continue;
            }
            const int slot = it % kSlots;
            ok = it < kSlots ||
                 mbar_wait_bounded(&ctl.empty[slot], static_cast<uint32_t>(it / kSlots - 1) & 1u);
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (!ok) break;
            // (a last V tile that the request's end cuts goes to the cleaning warp first, which
            // then completes the slot's barrier)
            const bool last = kv && (c + 1) * kTile > p.n;
            uint64_t* bar = last ? &ctl.v_last[slot] : &ctl.full[slot];
            if (lane == 0) {
              if (last) {
                ctl.issued_v[slot] += 1;
              } else {
                ctl.issued = it + 1;
              }
              mbar_arrive_expect_tx(bar, boxes * kBoxRows * 256);
            }
            __syncwarp();
            if (mine)
              mma::tma_load_4d(base_addr + Sh::kRing + slot * kTileBytes + half * kHalfBytes +
                                   box * kBoxRows * 128,
                               kv ? &map_v : &map_k, 64 * half, tok % P, p.kvh, pg, bar, policy);
            __syncwarp();
          }
          if (ok && c == p.c0 && piece > 0) {  // Q, once the previous piece's scores are over
            ok = mbar_wait_bounded(&ctl.q_empty, (piece - 1) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == 0) load_rows();
            __syncwarp();
          }
        }
        ++piece;
        more = walk.next(prm, P, p);
      }
      if (!ok && lane == 0) give_up();
    } else if (warp == kMmaWarp) {
      // ======================= MMA issue ==================================================
      if (umma::elect()) {
      constexpr int kStep = kQuant ? kTile / 2 : kTile;  // tokens of one set of scores
      constexpr uint32_t kScores = umma::instruction(kTile, kStep, false);
      constexpr uint32_t kOutput = umma::instruction(kTile, kTile, true);
      int it0 = 0;  // ring tiles of the pieces before
      uint32_t piece = 0, used0 = 0, used1 = 0;  // products of each stream
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity & 1u); };
      auto tile_addr = [&](int i) { return base_addr + Sh::kRing + (i % kSlots) * kTileBytes; };
      auto wait_tile = [&](int i) { return wait(&ctl.full[i % kSlots], static_cast<uint32_t>(i / kSlots)); };
      bool ok = true, more = walk.next(prm, P, p);
      while (ok && more) {
        const bool two = two_tiles(p);
        const int chunks = p.c1 - p.c0;
        // S_s = Q_tile K_c^T (int8: tokens 64 half .. of it); then the tile and Q are done with
        auto scores = [&](int s, int c, int half) {
          const uint32_t q = umma::operand(base_addr + Sh::kQ + (two ? s : 0) * kTileBytes, 16);
          const uint32_t k = umma::operand(tile_addr(it0 + 2 * c) + half * kStep * 128, 16);
          const uint32_t d = s_col(s) + half * kStep;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t off = ((j >> 2) * kHalfBytes + (j & 3) * 32) >> 4;
            umma::mma_ss(d, q + off, k + off, kScores, j > 0);
          }
          umma::commit(&ctl.s_full[kQuant ? 2 * s + half : s]);
          if ((!two || s == 1) && (!kQuant || half == 1)) {
            umma::commit(&ctl.empty[(it0 + 2 * c) % kSlots]);
            if (c == chunks - 1) umma::commit(&ctl.q_empty);
          }
        };
        ok = wait(&ctl.q_full, piece);
        ++piece;
        // the first scores of both streams
        for (int s = 0; s < 2 && ok; ++s) {
          const int c = two ? 0 : s;
          if (c >= chunks) break;
          if (s == 0 || !two) ok = wait_tile(it0 + 2 * c);
          for (int half = 0; half < (kQuant ? 2 : 1) && ok; ++half) scores(s, c, half);
        }
        more = walk.next(prm, P, p);  // (ahead: its look-ups wait for memory)
        for (int c = 0; c < chunks && ok; ++c) {
          const int s_begin = two ? 0 : c & 1, s_end = two ? 2 : s_begin + 1;
          const uint32_t v = umma::operand(tile_addr(it0 + 2 * c + 1), kHalfBytes);
          const bool first = two ? c == 0 : c < 2;  // of the piece in this stream
          const int next = two ? c + 1 : c + 2;
          if constexpr (kQuant) {
            for (int i = 0; i < 2 * (s_end - s_begin) && ok; ++i) {  // stream by stream, half by half
              const int half = two ? i >> 1 : i, s = two ? i & 1 : s_begin;
              const bool last = i == 2 * (s_end - s_begin) - 1;
              ok = wait(&ctl.p_ready[2 * s + half], s == 0 ? used0 : used1);
              if (ok && i == 0) ok = wait_tile(it0 + 2 * c + 1);
              if (!ok) break;
              if (half == 1) (s == 0 ? used0 : used1) += 1;
              const uint32_t d = o_col(s), a = s_col(s) + half * kStep;
              const uint32_t v0 = v + (half * kStep * 128 >> 4);
              umma::fence_after();
#pragma unroll
              for (int j = 0; j < 4; ++j)
                umma::mma_ts(d, a + 8 * j, v0 + j * (2048 >> 4), kOutput, !first || half > 0 || j > 0);
              umma::commit(&ctl.pv_done[s]);
              if (last) umma::commit(&ctl.empty[(it0 + 2 * c + 1) % kSlots]);
              if (next >= chunks) {
                if (half == 1) umma::commit(&ctl.o_full[s]);
              } else if (two) {
                if (i == 0) ok = wait_tile(it0 + 2 * next);
                if (ok) scores(s, next, half);
              } else if (last) {
                // (one tile: two chunks ahead, whose K takes the ring tile that V just left)
                ok = wait_tile(it0 + 2 * next);
                if (ok) scores(s, next, 0);
                if (ok) scores(s, next, 1);
              }
            }
          }
          for (int s = s_begin; !kQuant && s < s_end && ok; ++s) {
            const uint32_t use = s == 0 ? used0++ : used1++;
            ok = wait(&ctl.p_half[s], use);
            if (ok && s == s_begin) ok = wait_tile(it0 + 2 * c + 1);
            if (!ok) break;
            const uint32_t d = o_col(s), a = s_col(s);
            // 16 tokens a step: 8 columns of P, 16 rows (2 KiB) of V
            umma::fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              umma::mma_ts(d, a + 8 * j, v + j * (2048 >> 4), kOutput, !first || j > 0);
            ok = wait(&ctl.p_ready[s], use);
            if (!ok) break;
            umma::fence_after();
#pragma unroll
            for (int j = 4; j < 8; ++j)
              umma::mma_ts(d, a + 8 * j, v + j * (2048 >> 4), kOutput, true);
            if (s == s_end - 1) umma::commit(&ctl.empty[(it0 + 2 * c + 1) % kSlots]);
            if (next >= chunks) umma::commit(&ctl.o_full[s]);
            if (next < chunks) {
              if (s == s_begin) ok = wait_tile(it0 + 2 * next);
              if (ok) scores(s, next, 0);
            }
          }
        }
        it0 += 2 * chunks;
      }
      if (!ok) {
        give_up();
        umma::commit(&ctl.drained);  // what was issued must be over before the memory is freed
        wait(&ctl.drained, 0);
      }
      }
      __syncwarp();
    } else if (!kQuant && warp == kCleanWarp) {
      // ======================= V rows past the last token ===================================
      int it = 0;
      uint32_t cleaned = 0;  // bit per ring tile: parity of its uses
      while (walk.next(prm, P, p)) {
        it += 2 * (p.c1 - p.c0);
        const int valid = p.n - (p.c1 - 1) * kTile;  // tokens of the last chunk
        if (valid >= kTile) continue;
        const int slot = (it - 1) % kSlots;
        // (this waits for all of the work before that tile, so the limit starts anew as long as
        // tiles are issued)
        bool ok = false;
        for (int before = -1; !ok;) {
          const int now = *static_cast<volatile int*>(&ctl.issued);
          if (now == before || *abort_flag) break;
          before = now;
          ok = mbar_wait_bounded(&ctl.v_last[slot], (cleaned >> slot) & 1u);
        }
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) give_up();
          break;
        }
        cleaned ^= 1u << slot;
        unsigned char* rows = smem + Sh::kRing + slot * kTileBytes;
        for (int u = valid * 8 + lane; u < kTile * 8; u += 32) {
          *reinterpret_cast<uint4*>(rows + u * 16) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(rows + kHalfBytes + u * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mma::mbar_arrive(&ctl.full[slot]);
      }
      __syncwarp();
    }
  }
  trigger_dependents();
  __syncwarp();
  __syncthreads();  // every load from tensor memory is over
  if (*abort_flag && tid == 0) {
    // copies in flight must land before the block's memory is given up
    const int issued = *static_cast<volatile int*>(&ctl.issued);
    constexpr int kInFlight = kQuant ? kRawSlots : kSlots;
    uint64_t* landed = kQuant ? ctl.raw_full : ctl.full;
    for (int i = max(0, issued - kInFlight); i < issued; ++i)
      mbar_wait_bounded(&landed[i % kInFlight], static_cast<uint32_t>(i / kInFlight) & 1u);
    for (int i = 0; i < kSlots; ++i) {
      const int uses = *static_cast<volatile int*>(&ctl.issued_v[i]);
      if (uses > 0) mbar_wait_bounded(&ctl.v_last[i], static_cast<uint32_t>(uses - 1) & 1u);
    }
    const int issued_q = *static_cast<volatile int*>(&ctl.issued_q);
    if (issued_q > 0) mbar_wait_bounded(&ctl.q_full, static_cast<uint32_t>(issued_q - 1) & 1u);
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

template <int P, int kTiles, bool kQuant>
cudaError_t launch_one(const TreeParams& p, int group, cudaStream_t stream, bool use_pdl) {
  CUtensorMap mq, mk, mv;
  cudaError_t e = encode_q_map(&mq, p, group);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (Q)");
  e = mma::encode_pool_map(&mk, p.k_cache, kQuant, p.num_pages, p.num_kv_heads, P);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (K)");
  e = mma::encode_pool_map(&mv, p.v_cache, kQuant, p.num_pages, p.num_kv_heads, P);
  if (e != cudaSuccess) return fail_at(e, "tensor map encode (V)");
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(tree_mma_kernel<P, kTiles, kQuant>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shared<kTiles, kQuant>::kBytes);
    if (e != cudaSuccess) return fail_at(e, "shared-memory attribute");
    configured.fetch_or(bit);
  }
  return fail_at(launch_kernel(tree_mma_kernel<P, kTiles, kQuant>, dim3(p.blocks), dim3(Roles<kQuant>::kThreads),
                               static_cast<size_t>(Shared<kTiles, kQuant>::kBytes), stream, use_pdl, mq, mk, mv, p),
                 "cudaLaunchKernelEx");
}

template <bool kQuant>
cudaError_t launch(const TreeParams& p, int group, int page_size, cudaStream_t stream, bool use_pdl) {
  const bool one = group * p.max_q_len <= kTile;
#define PA_TREE_CASE(P)                                                       \
  case P:                                                                     \
    return one ? launch_one<P, 1, kQuant>(p, group, stream, use_pdl)          \
               : launch_one<P, 2, kQuant>(p, group, stream, use_pdl);
  switch (page_size) {
    PA_TREE_CASE(16)
    PA_TREE_CASE(32)
    PA_TREE_CASE(64)
    PA_TREE_CASE(128)
  }
#undef PA_TREE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace tree
}  // namespace pa

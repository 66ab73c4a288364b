// Eviction by accumulated weight: which rows of each (request, kv head) stay, and the move
// of the kept rows to the front in order.
//
// Selection (select_kernel, one block per (request, kv head)).  The kept set is the first
// and the newest positions and, of the others, the `need` largest weights.  A weight maps
// to a 32-bit key that orders like it; the need-th largest key is found digit by digit from
// the top (11 + 11 + 10 bits: a histogram of the keys that share the digits found so far,
// then the bin in which the count from above reaches `need`).  Keys above it stay, of the
// equal ones the lowest positions.  Each thread owns a run of positions; two prefix sums over
// the threads (larger keys, equal keys) give every kept position its place.  Bound by the
// latency of a block's passes; the keys are read once and kept in shared memory.
//
// Move.  To other pages (compact_kernel): every row is independent.  In place
// (compact_in_place_kernel): kept[i] >= i, so moving in ascending batches never overwrites a
// row that is still to be read, as long as a batch is read whole before it is stored; a block
// owns one (request, kv head) and a slice of the channels of K or of V (slices do not touch
// one another's bytes, so they need no order).
// Bound by memory: the kept rows read and written once.  32 requests of 8K tokens to 2K rows
// (bf16, other pages) take 97 us for both, the move at 6.5 TB/s; one request 12.8 us, nine of
// them the selection.  In place 143 and 18.8 us: a block's batches follow one another.
#include <math_constants.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// ---- selection ------------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;  // two blocks an SM: 97 against 101 us for 32 requests of 8K
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kOwnBins = kBins / kSelectThreads;  // of a thread
// positions of a row whose keys stay in shared memory; longer rows read them again (from L2)
constexpr int kCachedKeys = 40 * 1024;

// Orders like the weight: larger weight, larger key; -0 equals 0; every NaN is the largest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const SelectParams p, int cached) {
  extern __shared__ __align__(16) uint32_t keys_s[];  // the keys, of rows of up to `cached`
  // the first digit has two histograms, for even and odd lanes: weights cluster in few
  // exponents, and a warp's counts of one bin queue up
  __shared__ int hist[4][kBins];
  __shared__ int warp_sums[3][kSelectWarps];
  __shared__ uint32_t found_s[3][2];  // digit, keys above it
  __shared__ int2 placed_s[kSelectWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const int ps = 31 - __clz(p.page_size);  // page sizes are powers of two
#pragma unroll
  for (int d = 0; d < 4; ++d)
    for (int i = tid; i < kBins; i += kSelectThreads) hist[d][i] = 0;
  grid_dependency_wait();
  trigger_dependents();  // (the move behind it waits for this grid's end)

  const int cap = p.max_seq_pages << ps;
  int n = p.cache_seqlens[b];
  if (n < 0 || n > cap) {
    if (tid == 0 && h == 0) record_error(p.err, kErrSeqLenOutOfRange);
    n = n < 0 ? 0 : cap;
  }
  const int count = min(n, p.budget);
  int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.num_kv_heads + h) * p.budget;
  if (h == 0 && tid == 0) p.new_seqlens[b] = count;
  for (int i = count + tid; i < p.budget; i += kSelectThreads) kept[i] = -1;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += kSelectThreads) kept[i] = i;
    return;
  }

  const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.page_table_stride;
  // Keys of positions j .. j + 3 (j a multiple of 4: one page, one 16-byte read; past n they are
  // whatever the page holds): from memory, or from shared memory for rows that fit it.
  auto keys_of = [&](int pg, int j) -> uint4 {
    if (pg < 0 || pg >= p.num_pages) {
      record_error(p.err, kErrPageOutOfRange);
      return make_uint4(0u, 0u, 0u, 0u);
    }
    const float4 w = *reinterpret_cast<const float4*>(
        p.weights + ((static_cast<int64_t>(pg) * p.num_kv_heads + h) << ps) + (j & (p.page_size - 1)));
    return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
  };
  constexpr int kAhead = 2;  // such reads on their way before the first is used
  const bool in_smem = n <= cached;
  auto read_keys = [&](uint4 (&k)[kAhead], int j, int step, bool memory) {
    int pg[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      k[u] = make_uint4(0u, 0u, 0u, 0u);
      pg[u] = 0;
      if (j + u * step < n) {
        if (memory) pg[u] = pt[(j + u * step) >> ps];
        else k[u] = *reinterpret_cast<const uint4*>(keys_s + j + u * step);
      }
    }
    if (memory) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j + u * step < n) k[u] = keys_of(pg[u], j + u * step);
    }
  };

  // candidates: neither among the first nor among the newest
  const int lo = p.num_first, hi = n - p.num_recent;
  int need = p.budget - p.num_first - p.num_recent;  // of the candidates; < hi - lo
  const bool none = need == 0;                        // only the first and the newest stay
  uint32_t prefix = 0;                                // digits of the need-th largest key
  __syncthreads();  // the histograms are clear
#pragma unroll
  for (int digit = 0; digit < 3; ++digit) {
    const int bits = digit < 2 ? 11 : 10, shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    if (none) break;
    int* bins = hist[digit == 0 ? lane & 1 : digit + 1];
    // (the keys come into shared memory with the first digit's pass)
    for (int j0 = 4 * tid; j0 < n; j0 += 4 * kAhead * kSelectThreads) {
      uint4 k[kAhead];
      read_keys(k, j0, 4 * kSelectThreads, digit == 0 || !in_smem);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = j0 + u * 4 * kSelectThreads;
        if (digit == 0 && in_smem && j < n) *reinterpret_cast<uint4*>(keys_s + j) = k[u];
        const uint32_t key[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e >= lo && j + e < hi && (digit == 0 || (key[e] >> (shift + bits)) == prefix))
            atomicAdd(&bins[(key[e] >> shift) & ((1u << bits) - 1u)], 1);
      }
    }
    __syncthreads();
    // bins from the largest down, kOwnBins a lane: the one in which the count from above
    // reaches `need`
    const int top = kBins - 1 - kOwnBins * tid;
    const int* sums = hist[digit == 0 ? 0 : digit + 1];
    int own[kOwnBins], total = 0;
#pragma unroll
    for (int i = 0; i < kOwnBins; ++i) {
      own[i] = sums[top - i] + (digit == 0 ? hist[1][top - i] : 0);
      total += own[i];
    }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) warp_sums[digit][warp] = incl;
    __syncthreads();
    int before = lane < warp ? warp_sums[digit][lane] : 0;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
    incl += before;
    int above = incl - total;
    if (above < need && incl >= need) {
      int i = 0;
#pragma unroll
      for (int u = 0; u < kOwnBins - 1; ++u)
        if (i == u && above + own[u] < need) {
          above += own[u];
          i = u + 1;
        }
      found_s[digit][0] = top - i;
      found_s[digit][1] = above;
    }
    __syncthreads();
    prefix = (prefix << bits) | found_s[digit][0];
    need -= static_cast<int>(found_s[digit][1]);
  }
  // `prefix` is the smallest kept key; `need` of the keys equal to it stay (the lowest
  // positions)

  // Each thread places the kept positions of its run, eight at a time; prefix sums over the
  // threads say where it starts.
  constexpr int kEight = 8;
  const int run = ((n + kSelectThreads - 1) / kSelectThreads + kEight - 1) / kEight * kEight;
  const int r0 = min(tid * run, n), r1 = min(n, r0 + run);
  auto load_run = [&](uint32_t (&k)[kEight], int j) {
    if (none) return;
    uint4 x[kAhead];
    read_keys(x, j, 4, !in_smem);
    k[0] = x[0].x; k[1] = x[0].y; k[2] = x[0].z; k[3] = x[0].w;
    k[4] = x[1].x; k[5] = x[1].y; k[6] = x[1].z; k[7] = x[1].w;
  };
  auto judge = [&](int j, uint32_t k, bool& keep, bool& tie) {
    const bool in = j < r1;
    const bool always = j < lo || j >= hi;
    keep = in && (always || (!none && k > prefix));
    tie = in && !always && !none && k == prefix;
  };
  int sure = 0, equal = 0;  // this thread's
  for (int j = r0; j < r1; j += kEight) {
    uint32_t k[kEight];
    load_run(k, j);
#pragma unroll
    for (int u = 0; u < kEight; ++u) {
      bool keep, tie;
      judge(j + u, k[u], keep, tie);
      sure += keep;
      equal += tie;
    }
  }
  int sure_at = sure, equal_at = equal;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sure_at, d), eq = __shfl_up_sync(0xffffffffu, equal_at, d);
    if (lane >= d) {
      sure_at += up;
      equal_at += eq;
    }
  }
  if (lane == 31) placed_s[warp] = make_int2(sure_at, equal_at);
  __syncthreads();
  int2 other = make_int2(0, 0);
  if (lane < warp) other = placed_s[lane];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    other.x += __shfl_xor_sync(0xffffffffu, other.x, d);
    other.y += __shfl_xor_sync(0xffffffffu, other.y, d);
  }
  sure_at += other.x - sure;
  equal_at += other.y - equal;
  for (int j = r0; j < r1; j += kEight) {
    uint32_t k[kEight];
    load_run(k, j);
#pragma unroll
    for (int u = 0; u < kEight; ++u) {
      bool keep, tie;
      judge(j + u, k[u], keep, tie);
      if (keep || (tie && equal_at < need)) kept[sure_at + min(equal_at, need)] = j + u;
      sure_at += keep;
      equal_at += tie;
    }
  }
}

// ---- the move -------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;

// Pool row of position j of the request, -1 where its page is outside the pool.
__device__ __forceinline__ int64_t pool_row(const CompactParams& p, const int32_t* table, int j,
                                            int h) {
  const int ps = 31 - __clz(p.page_size);  // page sizes are powers of two
  const int pg = table[j >> ps];
  if (pg < 0 || pg >= p.num_pages) {
    record_error(p.err, kErrPageOutOfRange);
    return -1;
  }
  return ((static_cast<int64_t>(pg) * p.num_kv_heads + h) << ps) + (j & (p.page_size - 1));
}

struct Move {
  int64_t src, dst;  // pool rows; src < 0: nothing moves
};

struct Row {  // what a block's (request, kv head) moves
  const int32_t *kept, *src_table, *dst_table;
  int n, first, count;
};

__device__ __forceinline__ Row row_of(const CompactParams& p, int b, int h) {
  Row r;
  r.kept = p.kept + (static_cast<int64_t>(b) * p.kept_heads + (p.kept_heads == 1 ? 0 : h)) * p.kept_stride;
  r.src_table = p.page_table + static_cast<int64_t>(b) * p.page_table_stride;
  r.dst_table = p.dst_page_table + static_cast<int64_t>(b) * p.dst_page_table_stride;
  r.n = max(0, min(p.cache_seqlens[b], p.max_seq_pages * p.page_size));
  r.first = p.begin != nullptr ? p.begin[b] : 0;
  r.count = max(0, min(p.counts[b], p.max_kept));
  return r;
}

template <bool kInPlace>
__device__ __forceinline__ Move move_of(const CompactParams& p, const Row& r, int i, int h) {
  Move m = {-1, -1};
  if (i >= r.count) return m;
  const int j = r.kept[i];
  const int64_t to = static_cast<int64_t>(r.first) + i;
  if (j < 0 || j >= r.n || to < 0 || to >= static_cast<int64_t>(p.dst_max_pages) * p.page_size ||
      (kInPlace && j < to)) {
    record_error(p.err, kErrKeptOutOfRange);
    return m;
  }
  if (kInPlace && j == to) return m;
  m.dst = pool_row(p, r.dst_table, static_cast<int>(to), h);
  if (m.dst >= 0) m.src = pool_row(p, r.src_table, j, h);
  return m;
}

// kPieces: 16-byte pieces of a row (16: bf16, 8: int8).  A warp moves 32 rows: each lane looks
// one up (kept position, both pages) and moves its 4-byte values, then the warp moves the
// rows themselves, 32 / kPieces at a time and four such steps in flight.
template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  constexpr int kAtOnce = 32 / kPieces;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z;
  grid_dependency_wait();
  const Row r = row_of(p, b, h);
  if (p.new_seqlens != nullptr && blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    p.new_seqlens[b] = r.first + r.count;
  const int i0 = (blockIdx.x * (kMoveThreads / 32) + warp) * 32;
  if (i0 >= r.count) return;
  const Move m = move_of<false>(p, r, i0 + lane, h);
  const int piece = lane % kPieces, sub = lane / kPieces;
  const uint4* k_in = static_cast<const uint4*>(p.k_cache) + piece;
  const uint4* v_in = static_cast<const uint4*>(p.v_cache) + piece;
  uint4* k_out = static_cast<uint4*>(p.k_cache) + piece;
  uint4* v_out = static_cast<uint4*>(p.v_cache) + piece;
  float w = 0.f, ks = 0.f, vs = 0.f;
  if (m.src >= 0) {
    if (p.weights != nullptr) w = p.weights[m.src];
    if (p.k_scale != nullptr) {
      ks = p.k_scale[m.src];
      vs = p.v_scale[m.src];
    }
  }
#pragma unroll
  for (int j = 0; j < 32; j += kAtOnce * kUnroll) {
    int64_t src[kUnroll], dst[kUnroll];
    uint4 k[kUnroll], v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      src[u] = __shfl_sync(0xffffffffu, m.src, j + u * kAtOnce + sub);
      dst[u] = __shfl_sync(0xffffffffu, m.dst, j + u * kAtOnce + sub);
      if (src[u] >= 0) {
        k[u] = k_in[src[u] * kPieces];
        v[u] = v_in[src[u] * kPieces];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (src[u] >= 0) {
        k_out[dst[u] * kPieces] = k[u];
        v_out[dst[u] * kPieces] = v[u];
      }
  }
  if (m.src >= 0) {
    if (p.weights != nullptr) p.weights[m.dst] = w;
    if (p.k_scale != nullptr) {
      p.k_scale[m.dst] = ks;
      p.v_scale[m.dst] = vs;
    }
  }
}

// In place.  blockIdx.x: slice s of kSlices * 2 (K slices, then V slices) of 4 pieces each.
template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads) compact_in_place_kernel(const CompactParams p) {
  constexpr int kSlicePieces = 4, kSlices = kPieces / kSlicePieces;
  constexpr int kRows = kMoveThreads / kSlicePieces;
  constexpr int kBatch = kRows * kUnroll;
  const int h = blockIdx.y, b = blockIdx.z;
  const bool is_v = blockIdx.x >= kSlices;
  const int piece = (blockIdx.x % kSlices) * kSlicePieces + threadIdx.x % kSlicePieces;
  const int lane_row = threadIdx.x / kSlicePieces;
  uint4* pool = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache);
  // the 4-byte values that travel with a row: the scale with its tensor's first slice, the
  // weight with V's first slice
  float* scale = blockIdx.x % kSlices == 0 ? (is_v ? p.v_scale : p.k_scale) : nullptr;
  float* weight = blockIdx.x == kSlices ? p.weights : nullptr;
  grid_dependency_wait();
  const Row r = row_of(p, b, h);
  if (p.new_seqlens != nullptr && blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    p.new_seqlens[b] = r.first + r.count;

  const bool carries = threadIdx.x % kSlicePieces == 0;
  for (int i0 = 0; i0 < r.count; i0 += kBatch) {
    Move m[kUnroll];
    uint4 x[kUnroll];
    float s[kUnroll], w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) m[u] = move_of<true>(p, r, i0 + u * kRows + lane_row, h);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (m[u].src >= 0) {
        x[u] = pool[m[u].src * kPieces + piece];
        if (carries && scale != nullptr) s[u] = scale[m[u].src];
        if (carries && weight != nullptr) w[u] = weight[m[u].src];
      }
    __syncthreads();  // the batch has been read: its targets may be overwritten
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (m[u].src >= 0) {
        pool[m[u].dst * kPieces + piece] = x[u];
        if (carries && scale != nullptr) scale[m[u].dst] = s[u];
        if (carries && weight != nullptr) weight[m[u].dst] = w[u];
      }
  }
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream, bool use_pdl) {
  const int64_t tokens = static_cast<int64_t>(p.max_seq_pages) * p.page_size;
  // (a table wider than that still holds short rows)
  const int cached = static_cast<int>(tokens < kCachedKeys ? tokens : kCachedKeys);
  const size_t smem = static_cast<size_t>(cached) * 4;
  if (smem > 14 * 1024) {  // 33 KiB of static shared memory are in the 48 that need no asking
    cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kCachedKeys * 4);
    if (e != cudaSuccess) return fail_at(e, "shared-memory attribute");
  }
  return fail_at(launch_kernel(select_kernel, dim3(p.num_kv_heads, p.bs), dim3(kSelectThreads), smem,
                               stream, use_pdl, p, cached),
                 "cudaLaunchKernelEx (selection)");
}

cudaError_t launch_compact(const CompactParams& p, bool int8, bool in_place, cudaStream_t stream,
                           bool use_pdl) {
  const int pieces = int8 ? 8 : 16;
  const unsigned hkv = static_cast<unsigned>(p.num_kv_heads), bs = static_cast<unsigned>(p.bs);
  if (in_place) {
    const dim3 grid(2 * pieces / 4, hkv, bs);
    return fail_at(launch_kernel(int8 ? compact_in_place_kernel<8> : compact_in_place_kernel<16>, grid,
                                 dim3(kMoveThreads), 0, stream, use_pdl, p),
                   "cudaLaunchKernelEx (move)");
  }
  const int blocks = (p.max_kept + kMoveThreads - 1) / kMoveThreads;  // 32 rows a warp
  const dim3 grid(static_cast<unsigned>(blocks > 0 ? blocks : 1), hkv, bs);
  return fail_at(launch_kernel(int8 ? compact_kernel<8> : compact_kernel<16>, grid, dim3(kMoveThreads),
                               0, stream, use_pdl, p),
                 "cudaLaunchKernelEx (move)");
}

}  // namespace pa

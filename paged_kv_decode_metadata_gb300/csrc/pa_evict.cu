// Eviction by accumulated weight: which rows of each (request, kv head) stay, and the move
// of the kept rows to the front in order.
//
// Selection (select_kernel, one block per (request, kv head)).  The kept set is the first
// and the newest positions and, of the others, the `need` largest weights.  A weight maps
// to a 32-bit key that orders like it; the need-th largest key is found digit by digit from
// the top (11 + 11 + 10 bits: a histogram of the keys that share the digits found so far,
// then the bin in which the count from above reaches `need`).  Keys above it stay, of the
// equal ones the lowest positions.  Each warp owns a run of positions; two prefix sums over
// the warps (larger keys, equal keys) give every kept position its place.  Bound by the
// latency of a block's passes; the keys are read once and kept in shared memory.
//
// Move.  To other pages (compact_kernel): a thread moves 16-byte pieces of K and V rows,
// every row independent.  In place (compact_in_place_kernel): kept[i] >= i, so moving in
// ascending batches never overwrites a row that is still to be read, as long as a batch is
// read whole before it is stored; a block owns one (request, kv head) and a slice of the
// channels of K or of V (slices do not touch one another's bytes, so they need no order).
// Bound by memory: the kept rows read and written once.
#include <math_constants.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// ---- selection ------------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
// positions whose keys stay in shared memory; longer rows read them again (from L2)
constexpr int kCachedKeys = 48 * 1024;

// Orders like the weight: larger weight, larger key; -0 equals 0; every NaN is the largest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive sum over the block, in thread order; *total gets the sum of all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += up;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += up;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v += warp_sums[warp - 1];
  *total = warp_sums[kSelectWarps - 1];
  __syncthreads();  // warp_sums may be used again
  return v;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p, int cached) {
  extern __shared__ uint32_t keys_s[];  // the first `cached` keys
  __shared__ int hist[kBins];
  __shared__ int warp_sums[kSelectWarps];
  __shared__ uint32_t found_s[2];  // digit, keys above it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const int P = p.page_size;
  grid_dependency_wait();

  const int cap = p.max_seq_pages * P;
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
  auto load_key = [&](int j) -> uint32_t {
    const int pg = pt[j / P];
    if (pg < 0 || pg >= p.num_pages) {
      record_error(p.err, kErrPageOutOfRange);
      return 0u;
    }
    return weight_key(p.weights[(static_cast<int64_t>(pg) * p.num_kv_heads + h) * P + j % P]);
  };
  auto key_at = [&](int j) -> uint32_t { return j < cached ? keys_s[j] : load_key(j); };
  const int in_smem = min(n, cached);
  for (int j = tid; j < in_smem; j += kSelectThreads) keys_s[j] = load_key(j);

  // candidates: neither among the first nor among the newest
  const int lo = p.num_first, hi = n - p.num_recent;
  int need = p.budget - p.num_first - p.num_recent;  // of the candidates; < hi - lo
  uint32_t prefix = 0;                                // digits of the need-th largest key
  int shift = 21;
#pragma unroll 1
  for (int digit = 0; digit < 3 && need > 0; ++digit) {
    const int bits = digit < 2 ? 11 : 10;
    for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    // (digit 0: no key has been narrowed yet; a 32-bit shift would be undefined)
    for (int j = lo + tid; j < hi; j += kSelectThreads) {
      const uint32_t k = key_at(j);
      if (digit == 0 || (k >> (shift + bits)) == prefix)
        atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    // bins from the largest down, two a thread: the one in which the count reaches `need`
    const int top = kBins - 1 - 2 * tid;
    const int c0 = hist[top], c1 = hist[top - 1];
    int all;
    const int incl = block_scan(c0 + c1, warp_sums, &all);
    const int above = incl - c0 - c1;
    if (above < need && incl >= need) {
      const bool first = above + c0 >= need;
      found_s[0] = first ? top : top - 1;
      found_s[1] = first ? above : above + c0;
    }
    __syncthreads();
    prefix = (prefix << bits) | found_s[0];
    need -= static_cast<int>(found_s[1]);
    shift -= digit == 0 ? 11 : 10;
    __syncthreads();
  }
  // `prefix` is the smallest kept key; `need` of the keys equal to it stay (the lowest
  // positions).  Nothing beyond the first and the newest is wanted when need was 0.
  const bool none = p.budget - p.num_first - p.num_recent == 0;

  // each warp places the kept positions of its run
  const int run = ((n + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int r0 = warp * run, r1 = min(n, r0 + run);
  int sure = 0, equal = 0;  // this warp's, over the run
  for (int j0 = r0; j0 < r1; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < r1;
    const bool cand = in && j >= lo && j < hi && !none;
    const uint32_t k = cand ? key_at(j) : 0u;
    const bool keep = in && (j < lo || j >= hi || (cand && k > prefix));
    sure += __popc(__ballot_sync(0xffffffffu, keep));
    equal += __popc(__ballot_sync(0xffffffffu, cand && k == prefix));
  }
  int total;
  const int sure_end = block_scan(lane == 0 ? sure : 0, warp_sums, &total);
  const int equal_end = block_scan(lane == 0 ? equal : 0, warp_sums, &total);
  int sure_at = __shfl_sync(0xffffffffu, sure_end, 0) - sure;
  int equal_at = __shfl_sync(0xffffffffu, equal_end, 0) - equal;
  const uint32_t below = (1u << lane) - 1u;
  for (int j0 = r0; j0 < r1; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < r1;
    const bool cand = in && j >= lo && j < hi && !none;
    const uint32_t k = cand ? key_at(j) : 0u;
    const bool keep = in && (j < lo || j >= hi || (cand && k > prefix));
    const bool tie = cand && k == prefix;
    const uint32_t keeps = __ballot_sync(0xffffffffu, keep), ties = __ballot_sync(0xffffffffu, tie);
    const int ties_before = equal_at + __popc(ties & below);
    const int place = sure_at + __popc(keeps & below) + min(ties_before, need);
    if (keep || (tie && ties_before < need)) kept[place] = j;
    sure_at += __popc(keeps);
    equal_at += __popc(ties);
  }
}

// ---- the move -------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;

// Pool row of position j of the request, -1 where its page is outside the pool.
__device__ __forceinline__ int64_t pool_row(const CompactParams& p, const int32_t* table, int j,
                                            int h) {
  const int page = j / p.page_size;
  const int pg = table[page];
  if (pg < 0 || pg >= p.num_pages) {
    record_error(p.err, kErrPageOutOfRange);
    return -1;
  }
  return (static_cast<int64_t>(pg) * p.num_kv_heads + h) * p.page_size + (j - page * p.page_size);
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

// kPieces: 16-byte pieces of a row (16: bf16, 8: int8).
template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  constexpr int kRows = kMoveThreads / kPieces;
  const int piece = threadIdx.x % kPieces, lane_row = threadIdx.x / kPieces;
  const int h = blockIdx.y, b = blockIdx.z;
  grid_dependency_wait();
  const Row r = row_of(p, b, h);
  if (p.new_seqlens != nullptr && blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    p.new_seqlens[b] = r.first + r.count;
  const int i0 = blockIdx.x * kRows * kUnroll + lane_row;
  if (blockIdx.x * kRows * kUnroll >= r.count) return;
  Move m[kUnroll];
  uint4 k[kUnroll], v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) m[u] = move_of<false>(p, r, i0 + u * kRows, h);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (m[u].src >= 0) {
      k[u] = static_cast<const uint4*>(p.k_cache)[m[u].src * kPieces + piece];
      v[u] = static_cast<const uint4*>(p.v_cache)[m[u].src * kPieces + piece];
    }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (m[u].src >= 0) {
      static_cast<uint4*>(p.k_cache)[m[u].dst * kPieces + piece] = k[u];
      static_cast<uint4*>(p.v_cache)[m[u].dst * kPieces + piece] = v[u];
      if (piece == 0 && p.weights != nullptr) p.weights[m[u].dst] = p.weights[m[u].src];
      if (piece == 1 && p.k_scale != nullptr) p.k_scale[m[u].dst] = p.k_scale[m[u].src];
      if (piece == 2 && p.v_scale != nullptr) p.v_scale[m[u].dst] = p.v_scale[m[u].src];
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
  const int cached = static_cast<int>(tokens < kCachedKeys ? tokens : kCachedKeys);
  const size_t smem = static_cast<size_t>(cached) * 4;
  if (smem > 32 * 1024) {
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
  const int rows = kMoveThreads / pieces * kUnroll;
  const int blocks = (p.max_kept + rows - 1) / rows;
  const dim3 grid(static_cast<unsigned>(blocks > 0 ? blocks : 1), hkv, bs);
  return fail_at(launch_kernel(int8 ? compact_kernel<8> : compact_kernel<16>, grid, dim3(kMoveThreads),
                               0, stream, use_pdl, p),
                 "cudaLaunchKernelEx (move)");
}

}  // namespace pa

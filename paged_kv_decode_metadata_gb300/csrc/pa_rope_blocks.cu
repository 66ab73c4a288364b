// Rotary positions on the new queries and keys, and the new keys and values written to a
// block-scaled cache (e4m3 codes, one power-of-two scale per block of tokens and head).
//
// Mathematics.  Angles as in pa_rope.cu: a 64-bit fraction of a turn per pair, times the position
// modulo 2^64.  A block's scale is the smallest power of two that brings its largest new value
// to 448 or less, or the scale it had where that is larger: growing by a power of two costs the
// codes that were there nothing but what falls below e4m3's range.
//
// Shape.  A thread block owns one scale block of one request (and a share of the heads), so the
// largest value is a reduction within it and no two write one scale.  Slot s of the grid is
// mapped to a request without a scan: request b's slots start at cu_seqlens_q[b] / B + 2 b,
// which leaves room for the blocks that its rows can touch, and a warp finds b by 32 probes a
// round.  8 lanes take a row, each with two 16-byte pieces that hold whole pairs, 32 rows at
// once; a thread keeps its token over all heads, so it computes its 8 sines once, keeps them in
// registers for the query heads and in its own places of shared memory for the keys.  Where requests
// have few new rows a warp has a block and a share of its heads.
//
// Bound by latency when decoding (32 requests, 32 / 8 heads: 4.3 us of dependent loads, a find, the
// sines and one round of rows) and by memory for prompts (8192 tokens: 39.6 us, 4.7 TB/s, 70 % of
// the copy rate: a block's chain of load, reduction, barrier and store for each head and 32 warps an
// SM leave gaps).
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kFewThreads = 128;

__device__ __forceinline__ void unpack(const uint4& w, float* x) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(v[i]);
    x[2 * i + 1] = bf16_hi(v[i]);
  }
}

__device__ __forceinline__ uint4 pack(const float* x) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Two values to e4m3 codes (round to even, saturated), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  return make_uint2(to_codes(x[0] * inv, x[1] * inv) | to_codes(x[2] * inv, x[3] * inv) << 16,
                    to_codes(x[4] * inv, x[5] * inv) | to_codes(x[6] * inv, x[7] * inv) << 16);
}

// Four codes times `ratio`, rounded to codes again.
__device__ __forceinline__ uint32_t rescale(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    out |= to_codes(lo * ratio, hi * ratio) << (16 * i);
  }
  return out;
}

// The smallest power of two s with top / s <= 448 = 1.75 * 2^8, at least 2^-126; 0 for top = 0.
__device__ __forceinline__ float needed_scale(float top) {
  if (!(top > 0.f)) return 0.f;
  const int bits = __float_as_int(top);
  const int e = ((bits >> 23) & 0xff) - 127 + ((bits & 0x7fffff) > 0x600000 ? -7 : -8);
  return __int_as_float((max(e, -126) + 127) << 23);
}

// Sine and cosine of `whole` 2^-31 half turns, to 1.4 ulp at most and half an ulp in general (a code
// that lies next to a border feels the steps that a plain fp32 sine is off).  The nearest quarter is
// taken off exactly; of the rest, |t| <= pi / 4, Taylor's series with the leading terms' rounding
// errors carried along: sin t = t + (t_lo - t^3 P(t^2)), cos t = (1 - u) + (.. - u_lo + t^4 Q(t^2)),
// u = t^2 / 2.
__device__ __forceinline__ void turn_of(int32_t whole, float& s, float& c) {
  const int32_t quarter = static_cast<int32_t>((static_cast<uint32_t>(whole) + (1u << 29)) >> 30);
  const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(whole) - (static_cast<uint32_t>(quarter) << 30));
  const float r = static_cast<float>(rest & ~0x3f), r_lo = static_cast<float>(rest & 0x3f);
  constexpr double kPi = 3.14159265358979323846 / 2147483648.0;
  constexpr float kHi = static_cast<float>(kPi), kLo = static_cast<float>(kPi - kHi);
  const float t = r * kHi;
  const float t_lo = fmaf(r_lo, kHi, fmaf(r, kLo, fmaf(r, kHi, -t)));
  const float t2 = t * t;
  float p = fmaf(t2, -1.f / 39916800.f, 1.f / 362880.f);
  p = fmaf(t2, p, -1.f / 5040.f);
  p = fmaf(t2, p, 1.f / 120.f);
  p = fmaf(t2, p, -1.f / 6.f);
  float sn = t + fmaf(t * t2, p, t_lo);
  float q = fmaf(t2, 1.f / 479001600.f, -1.f / 3628800.f);
  q = fmaf(t2, q, 1.f / 40320.f);
  q = fmaf(t2, q, -1.f / 720.f);
  q = fmaf(t2, q, 1.f / 24.f);
  const float u = 0.5f * t2, w = 1.f - u;
  const float u_lo = fmaf(t, t_lo, 0.5f * fmaf(t, t, -t2));
  float cs = w + (((1.f - w) - u) + fmaf(t2 * t2, q, -u_lo));
  if (quarter & 1) {
    const float x = sn;
    sn = cs;
    cs = -x;
  }
  s = quarter & 2 ? -sn : sn;
  c = quarter & 2 ? -cs : cs;
}

// A scale block that gets rows: the slot's request, its rows and where they go.
struct Block {
  int count;           // new rows
  int held;            // rows of the block before them
  int in_page;         // row of its page of the first new one
  int64_t page, t0;    // (page: 0 where the table's is outside the pool); the first new token
  bool cached;

  // Whole-warp.  False: nothing to do.
  __device__ __forceinline__ bool find(const RopeBlocksParams& p, int slot, int lane, bool report) {
    const int B = 1 << p.block_shift;
    int lo = 0, hi = p.bs;  // the last request whose slots start at or before this one
    while (true) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      // (a start outside [0, total_q] has a slot all the same, so that the request is refused there)
      const bool before =
          at < hi && (min(max(p.cu_seqlens_q[at], 0), p.total_q) >> p.block_shift) + 2 * at <= slot;
      const uint32_t miss = ~__ballot_sync(0xffffffffu, before);
      const int ahead = miss == 0 ? 32 : __ffs(miss) - 1;
      if (ahead == 0) return false;
      lo += (ahead - 1) * step;
      hi = min(hi, lo + step);
      if (step == 1) break;
    }
    const int b = lo;
    const int q_begin = p.cu_seqlens_q[b], q_len = p.cu_seqlens_q[b + 1] - q_begin;
    const int n = p.cache_seqlens[b];
    if (q_begin < 0 || q_len < 0 || q_len > p.max_q_len || q_begin > p.total_q - q_len || n < q_len ||
        n > p.max_seq_pages << p.page_shift) {
      if (report) record_error(p.err, kErrSeqLenOutOfRange);
      return false;
    }
    const int begin = n - q_len;
    const int block = (begin >> p.block_shift) + slot - ((q_begin >> p.block_shift) + 2 * b);
    const int first = max(block << p.block_shift, begin);
    count = min((block + 1) << p.block_shift, n) - first;
    if (count <= 0) return false;
    const int at = p.page_table[b * p.page_table_stride + (first >> p.page_shift)];
    cached = at >= 0 && at < p.num_pages;
    if (!cached && report) record_error(p.err, kErrPageOutOfRange);
    page = cached ? at : 0;
    in_page = first & ((1 << p.page_shift) - 1);
    held = first & (B - 1);
    t0 = static_cast<int64_t>(q_begin) + first - begin;
    return true;
  }
};

// A lane's two 16-byte pieces of a row, and their rotation.
template <bool kInterleaved>
struct Pieces {
  bool rotates;
  int a, b;
  __device__ __forceinline__ Pieces(int l, int half_pieces) : rotates(l < half_pieces) {
    a = kInterleaved || !rotates ? 2 * l : l;
    b = kInterleaved || !rotates ? 2 * l + 1 : l + half_pieces;
  }
  static __device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = kInterleaved ? 2 * i : i, v = kInterleaved ? 2 * i + 1 : i + 8;
      const float y0 = x[u], y1 = x[v];
      x[u] = y0 * c[i] - y1 * s[i];
      x[v] = y1 * c[i] + y0 * s[i];
    }
  }
};

__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const double turns = inv_freq * 0.15915494309189533577;  // / 2 pi
  return __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
}

// The sines of a token's pairs 8 l .. 8 l + 7.
__device__ __forceinline__ void sines_of(uint64_t position, const uint64_t* fraction, int l, float amplitude,
                                         float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    turn_of(static_cast<int32_t>((position * fraction[8 * l + k]) >> 32), s[k], c[k]);
    c[k] *= amplitude;
    s[k] *= amplitude;
  }
}

// kPasses: rows of a block, 32 at a time.
template <int kThreads, int kPasses, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kPasses <= 2 ? 1024 / kThreads : 2)
    rope_blocks_kernel(const RopeBlocksParams p) {
  constexpr int kRowsAtOnce = kThreads / 8;
  __shared__ uint64_t fraction[64];
  __shared__ float tops[2][kThreads / 32];
  extern __shared__ float4 sines[];  // [pass][chunk of two pairs][thread]
  const int tid = threadIdx.x, lane = tid & 31, l = tid & 7;
  const int half = p.rotary_dim / 2, half_pieces = p.rotary_dim / 16;
  grid_dependency_wait();

  Block blk;
  if (!blk.find(p, static_cast<int>(blockIdx.x), lane, tid == 0 && blockIdx.y == 0)) return;
  const int count = blk.count, held = blk.held, in_page = blk.in_page;
  const int64_t page = blk.page, t0 = blk.t0;

  // this share's heads
  const int parts = gridDim.y, part = blockIdx.y;
  const int q_from = static_cast<int>(static_cast<int64_t>(p.num_q_heads) * part / parts);
  const int q_to = static_cast<int>(static_cast<int64_t>(p.num_q_heads) * (part + 1) / parts);
  const int kv_from = static_cast<int>(static_cast<int64_t>(p.num_kv_heads) * part / parts);
  const int kv_to = static_cast<int>(static_cast<int64_t>(p.num_kv_heads) * (part + 1) / parts);

  const Pieces<kInterleaved> piece(l, half_pieces);
  const bool rotates = piece.rotates;
  const int pa = piece.a, pb = piece.b;
  // ----- the sines of a thread's tokens, and the query rows -------------------------------------
  // (four rows are on their way all the time: a row's place is filled again as it leaves)
  const int passes = (count + kRowsAtOnce - 1) / kRowsAtOnce, heads = q_to - q_from;
  constexpr int kDeep = 4;
  uint4 wa[kDeep], wb[kDeep];
  int ask_pass = 0, ask_head = 0;  // the row that is asked for next
  auto ask = [&](int u) {
    const int r = ask_pass * kRowsAtOnce + (tid >> 3);
    if (ask_pass < passes && r < count) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                        (t0 + r) * p.q_stride) + (q_from + ask_head) * 16;
      wa[u] = src[pa];
      wb[u] = src[pb];
    }
    if (++ask_head == heads) {
      ask_head = 0;
      ++ask_pass;
    }
  };
  if (heads > 0) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) ask(u);
  }
  if (half > 0) {
    if (tid < half) fraction[tid] = turn_fraction(p.inv_freq[tid]);
    __syncthreads();
  }
  float c[8], s[8];
  int pass = -1, head = heads;  // (the next row starts a pass)
  const int total = heads > 0 ? passes * heads : passes;
  for (int i = 0; i < total; i += kDeep) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (i + u >= total) break;
      if (heads == 0 || head == heads) {
        head = 0;
        ++pass;
        const int r = pass * kRowsAtOnce + (tid >> 3);
        if (rotates && r < count) {
          sines_of(static_cast<uint64_t>(p.positions[t0 + r]), fraction, l, p.amplitude, c, s);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            sines[(pass * 4 + k) * kThreads + tid] = make_float4(c[2 * k], s[2 * k], c[2 * k + 1], s[2 * k + 1]);
        }
      }
      if (heads == 0) continue;
      const int r = pass * kRowsAtOnce + (tid >> 3);
      if (r < count) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + (t0 + r) * p.q_out_stride) +
                     (q_from + head) * 16;
        if (rotates) {
          float x[16];
          unpack(wa[u], x);
          unpack(wb[u], x + 8);
          piece.turn(x, c, s);
          wa[u] = pack(x);
          wb[u] = pack(x + 8);
        }
        dst[pa] = wa[u];
        dst[pb] = wb[u];
      }
      ++head;
      ask(u);
    }
  }
  if (!blk.cached) return;

  // ----- keys and values: a (head, K or V) at a time, the next one's rows on their way ----------
  const int blocks = 1 << (p.page_shift - p.block_shift);
  uint4 next[kPasses][2];
  auto fetch = [&](int unit) {
    const int h = kv_from + (unit >> 1);
    const bool is_v = unit & 1;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + h * 128;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int r = pass * kRowsAtOnce + (tid >> 3);
      if (r < count) {
        const uint4* row = reinterpret_cast<const uint4*>(base + (t0 + r) * stride);
        next[pass][0] = row[pa];
        next[pass][1] = row[pb];
      } else {
        next[pass][0] = next[pass][1] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  const int units = 2 * (kv_to - kv_from);
  if (units > 0) fetch(0);
  for (int unit = 0; unit < units; ++unit) {
    const int h = kv_from + (unit >> 1);
    const bool is_v = unit & 1;
    const int64_t head_row = (page * p.num_kv_heads + h) << p.page_shift;  // the page's first row
    float* scale_at = (is_v ? p.v_scale : p.k_scale) + (page * p.num_kv_heads + h) * blocks +
                      (in_page >> p.block_shift);
    const float old = held > 0 ? *scale_at : 0.f;
    float x[kPasses][16];
    float top = 0.f;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      unpack(next[pass][0], x[pass]);
      unpack(next[pass][1], x[pass] + 8);
    }
    if (unit + 1 < units) fetch(unit + 1);
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int r = pass * kRowsAtOnce + (tid >> 3);
      if (r < count) {
        if (rotates && !is_v) {
          float c[8], s[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 w = sines[(pass * 4 + i) * kThreads + tid];
            c[2 * i] = w.x;
            s[2 * i] = w.y;
            c[2 * i + 1] = w.z;
            s[2 * i + 1] = w.w;
          }
          piece.turn(x[pass], c, s);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[pass][i]));
      }
    }
    top = warp_max(top);
    if (lane == 0) tops[unit & 1][tid >> 5] = top;
    __syncthreads();  // (the other of the two rows of `tops` is free: every thread has passed it)
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, tops[unit & 1][w]);
    const float need = needed_scale(top);
    const float scale = held > 0 ? fmaxf(old, need) : need;
    unsigned char* codes = static_cast<unsigned char*>(is_v ? p.v_cache : p.k_cache) + (head_row + in_page) * 128;
    if (held > 0 && scale != old) {
      const float ratio = old / scale;
      uint4* rows = reinterpret_cast<uint4*>(codes - held * 128);
      for (int u = tid; u < held * 8; u += kThreads) {
        uint4 w = rows[u];
        w.x = rescale(w.x, ratio);
        w.y = rescale(w.y, ratio);
        w.z = rescale(w.z, ratio);
        w.w = rescale(w.w, ratio);
        rows[u] = w;
      }
    }
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int r = pass * kRowsAtOnce + (tid >> 3);
      if (r < count) {
        uint2* dst = reinterpret_cast<uint2*>(codes + r * 128);
        dst[pa] = codes8(x[pass], inv);
        dst[pb] = codes8(x[pass] + 8, inv);
      }
    }
    // (every thread read the old scale before the barrier above)
    if (tid == 0 && !(held > 0 && scale == old)) *scale_at = scale;
  }
}

// Few new rows a block (decoding, short drafts): a warp has the block and a share of its heads,
// kRows rows (one or four) of 4 / kRows heads at once, 8 lanes a row, kPasses times.  A block's
// largest value is a reduction over 8 kRows lanes.  Blocks with more rows than that take several
// rounds, and read keys and values twice.
template <int kRows, int kPasses, bool kInterleaved>
__global__ void __launch_bounds__(kFewThreads) rope_few_kernel(const RopeBlocksParams p, int slots, int parts) {
  constexpr int kUnits = 4 / kRows, kLanes = 8 * kRows;
  __shared__ uint64_t fraction[64];
  const int tid = threadIdx.x, lane = tid & 31, l = lane & 7;
  const int row = (lane >> 3) % kRows, unit = (lane >> 3) / kRows;
  const int half = p.rotary_dim / 2;
  grid_dependency_wait();
  if (tid < half) fraction[tid] = turn_fraction(p.inv_freq[tid]);
  __syncthreads();
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 32) + (tid >> 5);
  const int slot = static_cast<int>(task / parts), part = static_cast<int>(task - static_cast<int64_t>(slot) * parts);
  if (slot >= slots) return;
  Block blk;
  if (!blk.find(p, slot, lane, lane == 0 && part == 0)) return;
  const int q_from = static_cast<int>(static_cast<int64_t>(p.num_q_heads) * part / parts);
  const int q_to = static_cast<int>(static_cast<int64_t>(p.num_q_heads) * (part + 1) / parts);
  const int kv_from = static_cast<int>(static_cast<int64_t>(p.num_kv_heads) * part / parts);
  const int kv_to = static_cast<int>(static_cast<int64_t>(p.num_kv_heads) * (part + 1) / parts);
  const Pieces<kInterleaved> piece(l, p.rotary_dim / 16);
  const int rounds = (blk.count + kRows * kPasses - 1) / (kRows * kPasses);
  float c[kPasses][8], s[kPasses][8];
  auto sines = [&](int round) {
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int r = (round * kPasses + pass) * kRows + row;
      if (piece.rotates && r < blk.count)
        sines_of(static_cast<uint64_t>(p.positions[blk.t0 + r]), fraction, l, p.amplitude, c[pass], s[pass]);
    }
  };
  for (int round = 0; round < rounds; ++round) {
    sines(round);
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int r = (round * kPasses + pass) * kRows + row;
      if (r >= blk.count) continue;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (blk.t0 + r) * p.q_stride);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + (blk.t0 + r) * p.q_out_stride);
      for (int h = q_from + unit; h < q_to; h += kUnits) {
        uint4 wa = src[h * 16 + piece.a], wb = src[h * 16 + piece.b];
        if (piece.rotates) {
          float x[16];
          unpack(wa, x);
          unpack(wb, x + 8);
          piece.turn(x, c[pass], s[pass]);
          wa = pack(x);
          wb = pack(x + 8);
        }
        dst[h * 16 + piece.a] = wa;
        dst[h * 16 + piece.b] = wb;
      }
    }
  }
  if (!blk.cached) return;
  const int blocks = 1 << (p.page_shift - p.block_shift);
  const int units = 2 * (kv_to - kv_from);  // (head, K or V)
  for (int u0 = 0; u0 < units; u0 += kUnits) {
    const int u = u0 + unit;
    const bool live = u < units, is_v = u & 1;
    const int h = kv_from + (u >> 1);
    const int64_t head = blk.page * p.num_kv_heads + h;
    float* scale_at = (is_v ? p.v_scale : p.k_scale) + head * blocks + (blk.in_page >> p.block_shift);
    unsigned char* codes =
        static_cast<unsigned char*>(is_v ? p.v_cache : p.k_cache) + ((head << p.page_shift) + blk.in_page) * 128;
    const float old = live && blk.held > 0 ? *scale_at : 0.f;
    float x[kPasses][16];
    auto values = [&](int round) {  // the unit's rows of a round, turned
      if (rounds > 1) sines(round);
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int r = (round * kPasses + pass) * kRows + row;
        uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
        if (live && r < blk.count) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) +
                                                            (blk.t0 + r) * (is_v ? p.v_stride : p.k_stride) + h * 128);
          wa = src[piece.a];
          wb = src[piece.b];
        }
        unpack(wa, x[pass]);
        unpack(wb, x[pass] + 8);
        if (piece.rotates && !is_v && r < blk.count) piece.turn(x[pass], c[pass], s[pass]);
      }
    };
    float top = 0.f;
    for (int round = 0; round < rounds; ++round) {
      values(round);
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[pass][i]));
    }
#pragma unroll
    for (int d = kLanes / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float need = needed_scale(top);
    const float scale = blk.held > 0 ? fmaxf(old, need) : need;
    // blocks whose scale grows: the rows they held, by the whole warp
    const bool grows = live && blk.held > 0 && scale != old;
    uint32_t todo = __ballot_sync(0xffffffffu, grows && lane % kLanes == 0);
    while (todo != 0) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      const float ratio = __shfl_sync(0xffffffffu, old / scale, from);
      uint4* rows = reinterpret_cast<uint4*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(codes), from) -
          static_cast<unsigned long long>(blk.held) * 128);
      for (int i0 = lane; i0 < blk.held * 8; i0 += 4 * 32) {
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + 32 * k < blk.held * 8) w[k] = rows[i0 + 32 * k];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + 32 * k < blk.held * 8)
            rows[i0 + 32 * k] = make_uint4(rescale(w[k].x, ratio), rescale(w[k].y, ratio), rescale(w[k].z, ratio),
                                           rescale(w[k].w, ratio));
      }
    }
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) values(round);
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int r = (round * kPasses + pass) * kRows + row;
        if (live && r < blk.count) {
          uint2* dst = reinterpret_cast<uint2*>(codes + r * 128);
          dst[piece.a] = codes8(x[pass], inv);
          dst[piece.b] = codes8(x[pass] + 8, inv);
        }
      }
    }
    __syncwarp();  // (every lane has the old scale)
    if (live && lane % kLanes == 0 && !(blk.held > 0 && scale == old)) *scale_at = scale;
  }
}

template <int kThreads, int kPasses>
cudaError_t launch_many(const RopeBlocksParams& p, bool interleaved, int64_t slots, cudaStream_t stream, bool use_pdl) {
  // Few blocks of tokens: the heads over several thread blocks, down to one kv head each.
  const int most = p.num_kv_heads > p.num_q_heads / 4 ? p.num_kv_heads : p.num_q_heads / 4;
  int parts = 1;
  while (parts < most && slots * parts < 152 * 8) parts *= 2;
  if (parts > most) parts = most < 1 ? 1 : most;
  void (*kernel)(const RopeBlocksParams) =
      interleaved ? rope_blocks_kernel<kThreads, kPasses, true> : rope_blocks_kernel<kThreads, kPasses, false>;
  const size_t smem = p.rotary_dim > 0 ? static_cast<size_t>(kPasses) * 4 * kThreads * 16 : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return fail_at(e, "shared-memory attribute");
  }
  return fail_at(launch_kernel(kernel, dim3(static_cast<unsigned>(slots), static_cast<unsigned>(parts)),
                               dim3(kThreads), smem, stream, use_pdl, p),
                 "cudaLaunchKernelEx");
}

template <int kRows, int kPasses>
cudaError_t launch_few(const RopeBlocksParams& p, bool interleaved, int64_t slots, cudaStream_t stream, bool use_pdl) {
  // a warp down to four q rows and a kv head, while there are not two warps a scheduler
  const int most = p.num_kv_heads > p.num_q_heads / 4 ? p.num_kv_heads : p.num_q_heads / 4;
  int parts = 1;
  while (parts < most && slots * parts < 152 * 16) parts *= 2;
  if (parts > most) parts = most < 1 ? 1 : most;
  void (*kernel)(const RopeBlocksParams, int, int) =
      interleaved ? rope_few_kernel<kRows, kPasses, true> : rope_few_kernel<kRows, kPasses, false>;
  const int64_t blocks = (slots * parts + kFewThreads / 32 - 1) / (kFewThreads / 32);
  return fail_at(launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads), 0, stream, use_pdl, p,
                               static_cast<int>(slots), parts),
                 "cudaLaunchKernelEx (few)");
}

}  // namespace

cudaError_t launch_rope_blocks(const RopeBlocksParams& p, bool interleaved, cudaStream_t stream, bool use_pdl) {
  const int block = 1 << p.block_shift;
  const int64_t slots = (static_cast<int64_t>(p.total_q) >> p.block_shift) + 2 * static_cast<int64_t>(p.bs);
  // The most new rows that a request can have, as far as the host knows: up to 8 a warp has a block
  // (64 requests, 32 / 8 heads, scale blocks of 64: 4 rows each 6.4 us and 8 rows 8.5, by thread
  // blocks 10.1 and 10.5).  Where it does not know, one a request on average is taken for decoding;
  // more may be a prompt among decoding requests, whose blocks are long for a warp (31 with a row
  // and one with 200: 11.2 us by thread blocks, 57 by warps).  Where it knows more than 8, requests
  // without rows may stand beside a prompt (256 of which one has 200 rows and two have one: 16 us by
  // thread blocks, 56 and 115 by warps that take 8 rows or one at a time), or all may be decoding all the
  // same (25, 10 and 7.4 us): up to 16 rows, 8 at a time cost least at their worst (19 us, where thread
  // blocks take 25 and one at a time 31).
  const int most = p.max_q_len < p.total_q ? p.max_q_len : p.total_q;
  const bool known = p.max_q_len < p.total_q, sparse = p.total_q <= p.bs;
  if (most == 1 || (sparse && !known)) return launch_few<1, 1>(p, interleaved, slots, stream, use_pdl);
  if (most <= 4) return launch_few<4, 1>(p, interleaved, slots, stream, use_pdl);
  if (most <= 8 || (sparse && most <= 16)) return launch_few<4, 2>(p, interleaved, slots, stream, use_pdl);
  return block == 16   ? launch_many<128, 1>(p, interleaved, slots, stream, use_pdl)
         : block == 32 ? launch_many<256, 1>(p, interleaved, slots, stream, use_pdl)
         : block == 64 ? launch_many<256, 2>(p, interleaved, slots, stream, use_pdl)
                       : launch_many<256, 4>(p, interleaved, slots, stream, use_pdl);
}

}  // namespace pa

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
// registers for the query heads and in its own places of shared memory for the keys.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / 8;

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

// kPasses: rows of a block, 32 at a time.
template <int kPasses, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_blocks_kernel(const RopeBlocksParams p) {
  __shared__ uint64_t fraction[64];
  __shared__ float tops[2][kThreads / 32];
  extern __shared__ float4 sines[];  // [pass][chunk of two pairs][thread]
  const int tid = threadIdx.x, lane = tid & 31, l = tid & 7;
  const int half = p.rotary_dim / 2, half_pieces = p.rotary_dim / 16;
  grid_dependency_wait();

  // ----- the slot's request and block ---------------------------------------------------------
  const int slot = blockIdx.x, B = 1 << p.block_shift;
  int lo = 0, hi = p.bs;  // the last request whose slots start at or before this one
  bool found = true;
  while (found) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool before = at < hi && (p.cu_seqlens_q[at] >> p.block_shift) + 2 * at <= slot;
    const uint32_t miss = ~__ballot_sync(0xffffffffu, before);
    const int ahead = miss == 0 ? 32 : __ffs(miss) - 1;
    found = ahead > 0;
    lo += (ahead - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  if (!found) return;
  const int b = lo;
  const int q_begin = p.cu_seqlens_q[b], q_len = p.cu_seqlens_q[b + 1] - q_begin;
  const int n = p.cache_seqlens[b];
  if (q_begin < 0 || q_len < 0 || q_len > p.max_q_len || q_begin > p.total_q - q_len || n < q_len ||
      n > p.max_seq_pages << p.page_shift) {
    if (tid == 0 && blockIdx.y == 0) record_error(p.err, kErrSeqLenOutOfRange);
    return;
  }
  const int begin = n - q_len;
  const int block = (begin >> p.block_shift) + slot - ((q_begin >> p.block_shift) + 2 * b);
  const int first = max(block << p.block_shift, begin);
  const int count = min((block + 1) << p.block_shift, n) - first;  // new rows of this block
  if (count <= 0) return;
  const int page_in = p.page_table[b * p.page_table_stride + (first >> p.page_shift)];
  const bool cached = page_in >= 0 && page_in < p.num_pages;
  if (!cached && tid == 0 && blockIdx.y == 0) record_error(p.err, kErrPageOutOfRange);
  const int64_t page = cached ? page_in : 0;
  const int in_page = first & ((1 << p.page_shift) - 1);  // of the first new row
  const int held = first & (B - 1);                       // earlier rows of the block
  const int64_t t0 = static_cast<int64_t>(q_begin) + first - begin;

  // this share's heads
  const int parts = gridDim.y, part = blockIdx.y;
  const int q_from = static_cast<int>(static_cast<int64_t>(p.num_q_heads) * part / parts);
  const int q_to = static_cast<int>(static_cast<int64_t>(p.num_q_heads) * (part + 1) / parts);
  const int kv_from = static_cast<int>(static_cast<int64_t>(p.num_kv_heads) * part / parts);
  const int kv_to = static_cast<int>(static_cast<int64_t>(p.num_kv_heads) * (part + 1) / parts);

  if (half > 0) {
    if (tid < half) {
      const double turns = p.inv_freq[tid] * 0.15915494309189533577;  // / 2 pi
      fraction[tid] = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
    }
    __syncthreads();
  }
  const bool rotates = l < half_pieces;
  int pa, pb;  // this lane's two 16-byte pieces of a row
  if (kInterleaved || !rotates) {
    pa = 2 * l;
    pb = 2 * l + 1;
  } else {
    pa = l;
    pb = l + half_pieces;
  }
  auto turn = [&](float (&x)[16], const float (&c)[8], const float (&s)[8]) {
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[2 * i], y = x[2 * i + 1];
        x[2 * i] = a * c[i] - y * s[i];
        x[2 * i + 1] = y * c[i] + a * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[i], y = x[i + 8];
        x[i] = a * c[i] - y * s[i];
        x[i + 8] = y * c[i] + a * s[i];
      }
    }
  };

  // ----- the sines of a thread's tokens, and the query rows -------------------------------------
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int r = pass * kRowsAtOnce + (tid >> 3);
    if (r >= count) break;  // (no barrier below)
    const int64_t t = t0 + r;
    float c[8], s[8];
    if (rotates) {
      const uint64_t at = static_cast<uint64_t>(p.positions[t]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t phase = at * fraction[8 * l + i];
        // (24 bits of the angle's 32 are an exact fp32; the others turn the pair a little further:
        // a code that lies next to a border feels them)
        const int32_t whole = static_cast<int32_t>(phase >> 32);
        const float x = static_cast<float>(whole & ~0xff), rest = static_cast<float>(whole & 0xff) * 0x1.921fb6p-30f;
        float s0, c0;
        sincospif(x * 0x1p-31f, &s0, &c0);
        c[i] = fmaf(-s0, rest, c0) * p.amplitude;
        s[i] = fmaf(c0, rest, s0) * p.amplitude;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sines[(pass * 4 + i) * kThreads + tid] = make_float4(c[2 * i], s[2 * i], c[2 * i + 1], s[2 * i + 1]);
    }
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride);
    for (int h0 = q_from; h0 < q_to; h0 += 4) {
      uint4 wa[4], wb[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (h0 + u < q_to) {
          wa[u] = src[(h0 + u) * 16 + pa];
          wb[u] = src[(h0 + u) * 16 + pb];
        }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (h0 + u < q_to) {
          if (rotates) {
            float x[16];
            unpack(wa[u], x);
            unpack(wb[u], x + 8);
            turn(x, c, s);
            wa[u] = pack(x);
            wb[u] = pack(x + 8);
          }
          dst[(h0 + u) * 16 + pa] = wa[u];
          dst[(h0 + u) * 16 + pb] = wb[u];
        }
    }
  }
  if (!cached) return;

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
          turn(x[pass], c, s);
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

}  // namespace

cudaError_t launch_rope_blocks(const RopeBlocksParams& p, bool interleaved, cudaStream_t stream, bool use_pdl) {
  const int block = 1 << p.block_shift;
  const int64_t slots = (static_cast<int64_t>(p.total_q) >> p.block_shift) + 2 * static_cast<int64_t>(p.bs);
  // Few blocks of tokens: the heads over several thread blocks, down to one kv head each.
  const int most = p.num_kv_heads > p.num_q_heads / 4 ? p.num_kv_heads : p.num_q_heads / 4;
  int parts = 1;
  while (parts < most && slots * parts < 152 * 8) parts *= 2;
  if (parts > most) parts = most < 1 ? 1 : most;
#define PA_BLOCKS_CASE(PASSES) \
  (interleaved ? rope_blocks_kernel<PASSES, true> : rope_blocks_kernel<PASSES, false>)
  void (*kernel)(const RopeBlocksParams) = block <= 32   ? PA_BLOCKS_CASE(1)
                                           : block == 64 ? PA_BLOCKS_CASE(2)
                                                         : PA_BLOCKS_CASE(4);
#undef PA_BLOCKS_CASE
  const size_t smem = p.rotary_dim > 0 ? static_cast<size_t>(block <= 32 ? 1 : block / 32) * 4 * kThreads * 16 : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return fail_at(e, "shared-memory attribute");
  }
  return fail_at(launch_kernel(kernel, dim3(static_cast<unsigned>(slots), static_cast<unsigned>(parts)),
                               dim3(kThreads), smem, stream, use_pdl, p),
                 "cudaLaunchKernelEx");
}

}  // namespace pa

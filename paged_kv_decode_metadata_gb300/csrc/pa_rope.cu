// Rotary positions on the new queries and keys, and the new keys and values written to the
// paged cache (bf16, or int8 codes with a scale per row).
//
// Mathematics.  Pair i of a head turns by positions[t] * inv_freq[i] radians.  The angle is
// kept in turns: inv_freq / 2 pi becomes a 64-bit fraction of a turn once per thread block,
// and position times fraction modulo 2^64 is the fraction of the angle's last turn exactly
// (the integer product drops whole turns by itself), so far positions cost no accuracy and
// no 64-bit floating point per angle.  sincospif of that fraction is fp32 to 2 ulp.
//
// Layout.  A row (128 channels of one head) belongs to 8 lanes, each with two 16-byte
// pieces that hold whole pairs: pieces (l, l + R/16) of the half layout, (2l, 2l+1) of the
// interleaved one, with the pass-through pieces shared out over the remaining lanes.  Lane l
// turns pairs 8l .. 8l+7 either way.  The 64 sines and cosines of a token are computed once
// per block into shared memory.  int8 rows take their largest magnitude over the 8 lanes.
//
// Bound by memory (rows read once, written once) for prompts, by launch latency and the chain
// position -> sine -> rows for a decode step.
#include <utility>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRowLanes = 8;
constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / kRowLanes;

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(v[i]);
    x[2 * i + 1] = bf16_hi(v[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Eight codes: round to even of x / scale, largest magnitude 127.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = max(-127, min(127, __float2int_rn(x[i] * inv)));
    w[i >> 2] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

template <bool kInt8, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  __shared__ float2 turn[64];  // (cos, sin) * amplitude of each pair
  const int tid = threadIdx.x, l = tid & (kRowLanes - 1);
  const int half_pieces = p.rotary_dim / 16;
  grid_dependency_wait();

  const bool rotates = l < half_pieces;
  int pa, pb;  // this lane's two 16-byte pieces of a row
  if (kInterleaved || !rotates) {
    pa = 2 * l;
    pb = 2 * l + 1;
  } else {
    pa = l;
    pb = l + half_pieces;
  }
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int rows = hq + 2 * hkv;
  uint64_t fraction = 0;
  if (tid < p.rotary_dim / 2) {
    const double turns = p.inv_freq[tid] * 0.15915494309189533577;  // / 2 pi
    fraction = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
  }

  for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    __syncthreads();  // the previous token's sines have been used
    if (tid < p.rotary_dim / 2) {
      const uint64_t phase = static_cast<uint64_t>(p.positions[t]) * fraction;
      const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
      float s, c;
      sincospif(x, &s, &c);
      turn[tid] = make_float2(c * p.amplitude, s * p.amplitude);
    }
    const int64_t slot = p.slots[t];
    const bool cached = slot >= 0 && slot < p.num_pages * p.page_size;
    if (slot >= 0 && !cached && tid == 0 && blockIdx.y == 0)
      record_error(p.err, kErrSlotOutOfRange);
    const int64_t page = cached ? slot / p.page_size : 0;
    const int row_in_page = cached ? static_cast<int>(slot - page * p.page_size) : 0;
    __syncthreads();
    for (int r0 = blockIdx.y * kRowsAtOnce; r0 < rows; r0 += gridDim.y * kRowsAtOnce) {
      const int r = r0 + tid / kRowLanes;
      // (every lane of a row's 8 takes the same path; the int8 shuffles stay inside them)
      const bool live = r < rows && (r < hq || cached);
      const bool is_v = r >= hq + hkv;
      const int head = r < hq ? r : is_v ? r - hq - hkv : r - hq;
      uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
      if (live) {
        const __nv_bfloat16* src =
            r < hq ? static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride
                   : is_v ? static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride
                          : static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride;
        const uint4* row = reinterpret_cast<const uint4*>(src + static_cast<int64_t>(head) * 128);
        wa = row[pa];
        wb = row[pb];
      }
      float a[8], b[8];
      unpack8(wa, a);
      unpack8(wb, b);
      const bool turned = rotates && !is_v;
      if (turned) {
        if constexpr (kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 ca = turn[8 * l + i], cb = turn[8 * l + 4 + i];
            const float x0 = a[2 * i], x1 = a[2 * i + 1], y0 = b[2 * i], y1 = b[2 * i + 1];
            a[2 * i] = x0 * ca.x - x1 * ca.y;
            a[2 * i + 1] = x1 * ca.x + x0 * ca.y;
            b[2 * i] = y0 * cb.x - y1 * cb.y;
            b[2 * i + 1] = y1 * cb.x + y0 * cb.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = turn[8 * l + i];
            const float x = a[i], y = b[i];
            a[i] = x * cs.x - y * cs.y;
            b[i] = y * cs.x + x * cs.y;
          }
        }
      }
      if (r < hq) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) +
                                              t * p.q_out_stride + static_cast<int64_t>(head) * 128);
        dst[pa] = turned ? pack8(a) : wa;
        dst[pb] = turned ? pack8(b) : wb;
      }
      const int64_t dst_row = (page * hkv + head) * p.page_size + row_in_page;
      if constexpr (kInt8) {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
        for (int m = 1; m < kRowLanes; m <<= 1)
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
        if (live && r >= hq) {
          const float scale = big / 127.f;
          const float inv = scale > 0.f ? 1.f / scale : 0.f;
          uint2* dst = reinterpret_cast<uint2*>(static_cast<int8_t*>(is_v ? p.v_cache : p.k_cache) +
                                                dst_row * 128);
          dst[pa] = quantise8(a, inv);
          dst[pb] = quantise8(b, inv);
          if (l == 0) (is_v ? p.v_scale : p.k_scale)[dst_row] = scale;
        }
      } else if (live && r >= hq) {
        uint4* dst = reinterpret_cast<uint4*>(
            static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + dst_row * 128);
        dst[pa] = turned ? pack8(a) : wa;
        dst[pb] = turned ? pack8(b) : wb;
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool int8, bool interleaved, cudaStream_t stream,
                        bool use_pdl) {
  void (*kernel)(const RopeParams) = int8 ? (interleaved ? rope_kernel<true, true> : rope_kernel<true, false>)
                                          : (interleaved ? rope_kernel<false, true> : rope_kernel<false, false>);
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int groups = (rows + kRowsAtOnce - 1) / kRowsAtOnce;
  // few tokens: a block for every 32 rows of a token, so that all of them are in flight
  const dim3 grid(static_cast<unsigned>(p.num_tokens), p.num_tokens <= 1024 ? groups : 1);
  return launch_kernel(kernel, grid, dim3(kThreads), 0, stream, use_pdl, p);
}

}  // namespace pa

// Rotary positions on the new queries and keys, and the new keys and values written to the
// paged cache (bf16, or int8 codes with a scale per row).
//
// Mathematics.  Pair i of a head turns by positions[t] * inv_freq[i] radians.  The angle is
// kept in turns: inv_freq / 2 pi becomes a 64-bit fraction of a turn once per warp,
// and position times fraction modulo 2^64 is the fraction of the angle's last turn exactly
// (the integer product drops whole turns by itself), so far positions cost no accuracy and
// no 64-bit floating point per angle.  sincospif of that fraction is fp32 to 2 ulp.
//
// Layout.  A row (128 channels of one head) belongs to 8 lanes, each with two 16-byte
// pieces that hold whole pairs: pieces (l, l + R/16) of the half layout, (2l, 2l+1) of the
// interleaved one, with the pass-through pieces shared out over the remaining lanes.  Lane l
// turns pairs 8l .. 8l+7 either way.  A warp walks tokens by itself (no barrier): the fractions
// (64-bit floating point, slow here) once, the sines once a token.  int8 rows take their
// largest magnitude over the 8 lanes.
//
// Bound by memory (rows read once, written once) for prompts: 8192 tokens of 32 / 8 heads take
// 38.1 us in bf16 (5.3 TB/s, a last wave on 84 % of the places); by the sines before a token's
// rows where a warp has one token: 4097 tokens, int8, 64 / 8 heads, 36.5 us (4.4 TB/s); by the
// launch for a decode step: 32 tokens take 3.8 us, 3.4 of them on the host.
#include <utility>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRowLanes = 8;
constexpr int kThreads = 256;

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

// Eight codes: round to even of x lift inv, largest magnitude 127.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float lift, float inv) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = max(-127, min(127, __float2int_rn(x[i] * lift * inv)));
    w[i >> 2] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// A warp takes a token (a share of its rows where there are few tokens) at a time: lane group
// g of four has pairs 8 l + 2 g, + 1 of the token's sines, which every lane collects by
// shuffles, then rows go through four at a time, kDeep such steps in flight.
template <bool kInt8, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int parts) {
  constexpr int kDeep = 4;
  const int lane = threadIdx.x & 31, l = lane & (kRowLanes - 1), g = lane / kRowLanes;
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
  uint64_t fraction[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (rotates) {
      const double turns = p.inv_freq[8 * l + 2 * g + i] * 0.15915494309189533577;  // / 2 pi
      fraction[i] = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
    }
  const int steps = (rows + 3) / 4;                  // of four rows
  const int per_part = (steps + parts - 1) / parts;  // steps of a part of a token
  const int64_t tasks = static_cast<int64_t>(p.num_tokens) * parts;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  int64_t position = 0, slot = 0;
  if (task < tasks) {
    position = p.positions[task / parts];
    slot = p.slots[task / parts];
  }
  for (; task < tasks; task += stride) {
    const int64_t t = task / parts;
    const int part = static_cast<int>(task - t * parts);
    const int64_t at = position, to = slot;
    if (task + stride < tasks) {  // the next token's, ahead
      position = p.positions[(task + stride) / parts];
      slot = p.slots[(task + stride) / parts];
    }
    const bool cached = to >= 0 && to < p.num_pages * p.page_size;
    if (to >= 0 && !cached && lane == 0 && part == 0) record_error(p.err, kErrSlotOutOfRange);
    const int64_t page = cached ? to / p.page_size : 0;
    const int row_in_page = cached ? static_cast<int>(to - page * p.page_size) : 0;
    // (here, once a token: with its K rows below it cost the append 2 % even where it is off)
    if (p.weights != nullptr && cached && part == 0)
      for (int h = lane; h < hkv; h += 32) p.weights[(page * hkv + h) * p.page_size + row_in_page] = 0.f;
    float c[8], s[8];  // of pairs 8 l ..
    {
      float mine_c[2], mine_s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t phase = static_cast<uint64_t>(at) * fraction[i];
        const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
        sincospif(x, &mine_s[i], &mine_c[i]);
        mine_c[i] *= p.amplitude;
        mine_s[i] *= p.amplitude;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = __shfl_sync(0xffffffffu, mine_c[i & 1], (i >> 1) * kRowLanes + l);
        s[i] = __shfl_sync(0xffffffffu, mine_s[i & 1], (i >> 1) * kRowLanes + l);
      }
    }
    const int end = min(steps, (part + 1) * per_part);
    for (int step = part * per_part; step < end; step += kDeep) {
      uint4 wa[kDeep], wb[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int r = (step + u) * 4 + g;
        wa[u] = wb[u] = make_uint4(0u, 0u, 0u, 0u);
        if (step + u < end && r < rows) {
          const __nv_bfloat16* src =
              r < hq ? static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + r * 128
                     : r < hq + hkv ? static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride +
                                          (r - hq) * 128
                                    : static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride +
                                          (r - hq - hkv) * 128;
          const uint4* row = reinterpret_cast<const uint4*>(src);
          wa[u] = row[pa];
          wb[u] = row[pb];
        }
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        if (step + u >= end) break;  // (the whole warp)
        const int r = (step + u) * 4 + g;
        const bool live = r < rows && (r < hq || cached);
        const bool is_v = r >= hq + hkv;
        const int head = r < hq ? r : is_v ? r - hq - hkv : r - hq;
        float a[8], b[8];
        unpack8(wa[u], a);
        unpack8(wb[u], b);
        const bool turned = rotates && !is_v;
        if (turned) {
          if constexpr (kInterleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x0 = a[2 * i], x1 = a[2 * i + 1], y0 = b[2 * i], y1 = b[2 * i + 1];
              a[2 * i] = x0 * c[i] - x1 * s[i];
              a[2 * i + 1] = x1 * c[i] + x0 * s[i];
              b[2 * i] = y0 * c[4 + i] - y1 * s[4 + i];
              b[2 * i + 1] = y1 * c[4 + i] + y0 * s[4 + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x = a[i], y = b[i];
              a[i] = x * c[i] - y * s[i];
              b[i] = y * c[i] + x * s[i];
            }
          }
        }
        if (r < hq) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) +
                                                t * p.q_out_stride + static_cast<int64_t>(head) * 128);
          dst[pa] = turned ? pack8(a) : wa[u];
          dst[pb] = turned ? pack8(b) : wb[u];
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
            // (rows so small that 1 / scale would overflow are lifted by a power of two first)
            const float lift = big < 0x1p-60f ? 0x1p64f : 1.f;
            const float inv = scale > 0.f ? 1.f / (scale * lift) : 0.f;
            uint2* dst = reinterpret_cast<uint2*>(
                static_cast<int8_t*>(is_v ? p.v_cache : p.k_cache) + dst_row * 128);
            dst[pa] = quantise8(a, lift, inv);
            dst[pb] = quantise8(b, lift, inv);
            if (l == 0) (is_v ? p.v_scale : p.k_scale)[dst_row] = scale;
          }
        } else if (live && r >= hq) {
          uint4* dst = reinterpret_cast<uint4*>(
              static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + dst_row * 128);
          dst[pa] = turned ? pack8(a) : wa[u];
          dst[pb] = turned ? pack8(b) : wb[u];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool int8, bool interleaved, cudaStream_t stream,
                        bool use_pdl) {
  void (*kernel)(const RopeParams, int) =
      int8 ? (interleaved ? rope_kernel<true, true> : rope_kernel<true, false>)
           : (interleaved ? rope_kernel<false, true> : rope_kernel<false, false>);
  constexpr int kWarps = kThreads / 32;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  // Few tokens: a token's rows over several warps, up to one step of four rows each.
  const int steps = (rows + 3) / 4;
  int parts = 1;
  while (parts < steps && static_cast<int64_t>(p.num_tokens) * parts * 2 <= 152 * kWarps) parts *= 2;
  if (parts > steps) parts = steps;
  const int64_t warps = static_cast<int64_t>(p.num_tokens) * parts;
  const int64_t blocks = (warps + kWarps - 1) / kWarps, most = 152 * 4;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                       dim3(kThreads), 0, stream, use_pdl, p, parts);
}

}  // namespace pa

// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Mathematics.  At a node, its drafted children are tried in order: child x is accepted with
// probability w(x) / (S q(x)), where w is what is left of the target's row p after the children
// before it, max(p - c q, 0), and S its sum; a rejected child makes c += S.  (The residuals of
// residuals fold into one factor: max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0).)  With
// no draft probabilities a child was proposed for certain: w(x) / S, and a rejection takes w(x)
// out of w.  Where no child is left, the next token is drawn from w by inversion.  Whatever the
// draft proposed, tokens follow the target's distribution.
// Sums of w are integers (units of 2^-42), so they do not depend on the order, the number of
// threads or the split, and the token drawn is the same every time.  An fp32 weight becomes two
// 21-bit integers by two additions that round down.
//
// Shape.  A cluster of eight thread blocks has a request.  The children's p(x) and q(x) are
// gathered at once, so the walk down the tree is arithmetic, done by one warp of each block alike,
// which finds a node's next child by ballots.  Only a residual's sum needs a whole row (and the
// draft's): every block sums an eighth, a warp a contiguous piece of it, 512 tokens at a time; the
// block sums are exchanged through distributed shared memory, and the 512 tokens that hold the
// drawn number are read once more.  A chain needs one such row, the last node's.
//
// Bound by dependent latencies: the nodes, their probabilities, the row, the exchange, the batch once
// more.  One chain of four drafted tokens, vocabulary 32000: 5.5 us, about half of it launch; 32 of
// eight, 128000: 10.7 us in a graph, where their two rows' bytes would take 4.9.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// (256 threads: blocks of 512 and 1024 start more slowly than they save in rounds of loads, 32 chains
// at a vocabulary of 128000 11.7 and 12.6 us against 11.1; clusters of four as much)
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxNodes = 256;
constexpr float kUnits = 0x1p42f;  // a weight of 1
constexpr int kDeep = 4;           // loads of a row on their way: a batch of 4 x 128 tokens a warp
constexpr int kBatches = (1 << 20) / (kCluster * kWarps * kDeep * 128);  // of a warp's piece, at most

struct Shared {
  float p[kMaxNodes], q[kMaxNodes], u[kMaxNodes];
  long long token[kMaxNodes];
  int parent[kMaxNodes];
  int path[kMaxNodes];
  long long gone[kMaxNodes];  // without draft probabilities: tokens taken out of the row,
  float gone_p[kMaxNodes];    // and their probabilities
  unsigned long long batch_sum[kWarps][kBatches], warp_sum[kWarps], block_sum[2][kCluster];
  // what the walk has come to
  int node, length, num_gone;
  float c;   // w = max(p - c q, 0)
  int todo;  // 0: sum w for the next sibling, 1: draw the token
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Stores to the same variable of block `rank` of the cluster (which has started: that is waited for before
// the first of them).
__device__ __forceinline__ void store_remote(unsigned long long* at, uint32_t rank, unsigned long long v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(at)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}

// A weight in [0, 1] (NaN: 0) in units of 2^-42, rounded down: hi * 2^21 + lo.
__device__ __forceinline__ void to_units(float w, uint32_t& hi, uint32_t& lo) {
  const float t = fminf(fmaxf(w, 0.f), 1.f) * 0x1p21f;
  const float a = __fadd_rd(t, 0x1p23f);
  const float b = __fadd_rd((t - (a - 0x1p23f)) * 0x1p21f, 0x1p23f);
  hi = __float_as_uint(a) - 0x4b000000u;
  lo = __float_as_uint(b) - 0x4b000000u;
}

template <bool kVec>
__device__ __forceinline__ void load4(const float* row, int x, int vocab, float (&v)[4]) {
  if constexpr (kVec) {
    if (x < vocab) {  // (vocab is a multiple of 4)
      const float4 w = *reinterpret_cast<const float4*>(row + x);
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else {
      v[0] = v[1] = v[2] = v[3] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = x + j < vocab ? row[x + j] : 0.f;
  }
}

template <bool kVec>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    verify_kernel(const VerifyParams prm) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int b = blockIdx.y;
  // A block's memory may be stored to only once it runs: all arrive here, and wait before the walk.
  cluster_arrive();
  grid_dependency_wait();

  const int q_begin = prm.cu_seqlens_q[b];
  int q_len = prm.cu_seqlens_q[b + 1] - q_begin;
  if (q_begin < 0 || q_len < 0 || q_len > prm.max_q_len || q_begin > prm.total_q - q_len) {
    if (rank == 0 && tid == 0) record_error(prm.err, kErrSeqLenOutOfRange);
    q_len = 0;
  }
  const int n = prm.cache_seqlens != nullptr ? prm.cache_seqlens[b] : q_len;
  if (n < q_len) {
    if (rank == 0 && tid == 0) record_error(prm.err, kErrSeqLenOutOfRange);
    q_len = 0;
  }
  const int begin = n - q_len;
  int32_t* kept = prm.kept + static_cast<int64_t>(b) * prm.kept_stride;
  if (q_len == 0) {  // (the whole cluster)
    cluster_wait();
    if (rank == 0) {
      for (int i = tid; i < prm.max_q_len; i += kThreads) kept[i] = -1;
      if (tid == 0) {
        prm.counts[b] = 0;
        if (prm.begin != nullptr) prm.begin[b] = begin;
        prm.next_tokens[b] = -1;
      }
    }
    return;
  }

  // ----- the nodes and their probabilities --------------------------------------------------
  const int vocab = prm.vocab;
  if (tid < q_len) {
    int up = tid - 1;
    if (prm.parents != nullptr) {
      up = prm.parents[q_begin + tid];
      if (up < -1 || up >= tid) {
        if (rank == 0) record_error(prm.err, kErrTreeParent);
        up = -1;
      }
    }
    const long long x = prm.tokens[q_begin + tid];
    float p = 0.f, q = 1.f;
    if (tid > 0 && up >= 0) {
      if (x >= 0 && x < vocab) {
        p = prm.target_probs[(static_cast<int64_t>(q_begin) + up) * prm.target_stride + x];
        if (prm.draft_probs != nullptr)
          q = prm.draft_probs[(static_cast<int64_t>(q_begin) + up) * prm.draft_stride + x];
      } else if (rank == 0) {
        record_error(prm.err, kErrTokenOutOfRange);
      }
    }
    sh.parent[tid] = up;
    sh.token[tid] = x;
    sh.p[tid] = p;
    sh.q[tid] = q;
    sh.u[tid] = tid > 0 ? prm.uniforms[q_begin + tid] : 0.f;
  }
  __syncthreads();

  // a warp's piece of the row, and the eighth's
  const int piece = ((vocab + kCluster * kWarps - 1) / (kCluster * kWarps) + 127) / 128 * 128;
  const int64_t from64 = (static_cast<int64_t>(rank) * kWarps + warp) * piece;
  const int from = static_cast<int>(min(from64, static_cast<int64_t>(vocab)));
  const int to = static_cast<int>(min(from64 + piece, static_cast<int64_t>(vocab)));
  const float *p_row = nullptr, *q_row = nullptr;
  float c = 0.f;
  // units of the four weights at x; tokens that are gone count for nothing
  auto weights = [&](const float (&p)[4], const float (&q)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) to_units(q_row != nullptr ? fmaf(-c, q[j], p[j]) : p[j], hi[j], lo[j]);
  };
  // a batch's loads, all on their way at once
  auto load_batch = [&](int x0, float (&p)[kDeep][4], float (&q)[kDeep][4]) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int x = x0 + d * 128 + lane * 4;
      load4<kVec>(p_row, x, to, p[d]);
      if (q_row != nullptr) load4<kVec>(q_row, x, to, q[d]);
    }
  };
  auto warp_total = [](unsigned long long v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  // the sum of w over the row; batch, warp and block sums stay in shared memory
  auto row_sum = [&](int buffer) -> unsigned long long {
    unsigned long long total = 0;
    const int num_gone = sh.num_gone;
    for (int x0 = from, batch = 0; x0 < to; x0 += kDeep * 128, ++batch) {
      float p[kDeep][4], q[kDeep][4];
      load_batch(x0, p, q);  // (the next one's ahead of this one's sums: no faster)
      unsigned long long sum = 0;
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        uint32_t hi[4], lo[4];
        weights(p[d], q[d], hi, lo);
        sum += (static_cast<unsigned long long>(hi[0] + hi[1] + hi[2] + hi[3]) << 21) +
               (lo[0] + lo[1] + lo[2] + lo[3]);
      }
      for (int i = lane; i < num_gone; i += 32) {
        const long long x = sh.gone[i];
        if (x >= x0 && x < min(x0 + kDeep * 128, to)) {
          uint32_t hi, lo;
          to_units(sh.gone_p[i], hi, lo);
          sum -= (static_cast<unsigned long long>(hi) << 21) + lo;  // (of the whole warp's sum)
        }
      }
      sum = warp_total(sum);
      if (lane == 0) sh.batch_sum[warp][batch] = sum;
      total += sum;
    }
    if (lane == 0) sh.warp_sum[warp] = total;
    __syncthreads();
    if (tid < kCluster) {
      unsigned long long mine = 0;
      for (int w = 0; w < kWarps; ++w) mine += sh.warp_sum[w];
      store_remote(&sh.block_sum[buffer][rank], static_cast<uint32_t>(tid), mine);
    }
    cluster_arrive();
    cluster_wait();
    unsigned long long all = 0;
    for (int r = 0; r < kCluster; ++r) all += sh.block_sum[buffer][r];
    return all;
  };

  // ----- the walk: up to a residual that has to be summed, or to the end -----------------------
  int buffer = 0;
  unsigned long long all = 0;
  // (warp 0's, every lane alike)
  int next = 1, node = 0, length = 1, num_gone = 0;
  float walk_c = 0.f, sum = 1.f;  // w = max(p - c q, 0) and its sum, -1 where it is not known
  double left = 1.0;              // without draft probabilities: the row's sum less what is gone
  if (tid == 0) sh.path[0] = 0;
  cluster_wait();  // (every block of the cluster has started; the loads above took longer)
  while (true) {
    if (warp == 0) {
      const bool drafted = prm.draft_probs != nullptr;
      int todo = 1;
      for (int base = next & ~31; base < q_len && todo == 1; base += 32) {
        const int mine = base + lane;
        const int up = mine < q_len ? sh.parent[mine] : -1;
        const float my_p = mine < q_len ? sh.p[mine] : 0.f, my_q = mine < q_len ? sh.q[mine] : 0.f;
        const float my_u = mine < q_len ? sh.u[mine] : 0.f;
        const long long my_x = mine < q_len ? sh.token[mine] : -1;
        while (true) {  // the node's next child among these 32
          const uint32_t children = __ballot_sync(0xffffffffu, up == node && mine >= next);
          if (children == 0) break;
          const int at = __ffs(children) - 1;
          const float p = __shfl_sync(0xffffffffu, my_p, at), u = __shfl_sync(0xffffffffu, my_u, at);
          bool ok;
          if (drafted) {
            if (sum < 0.f) {  // (siblings before it were rejected)
              todo = 0;
              break;
            }
            const float q = __shfl_sync(0xffffffffu, my_q, at);
            const float w = walk_c > 0.f ? fmaxf(fmaf(-walk_c, q, p), 0.f) : p;
            ok = static_cast<double>(u) * static_cast<double>(q) * static_cast<double>(sum) < static_cast<double>(w);
            if (!ok) {
              walk_c += sum;
              sum = -1.f;
            }
          } else {
            const long long x = __shfl_sync(0xffffffffu, my_x, at);
            bool taken = false;
            for (int g = lane; g < num_gone; g += 32) taken = taken || sh.gone[g] == x;
            const float w = __any_sync(0xffffffffu, taken) ? 0.f : p;
            ok = static_cast<double>(u) * left < static_cast<double>(w);
            if (!ok && w > 0.f) {
              if (lane == 0) {
                sh.gone[num_gone] = x;
                sh.gone_p[num_gone] = p;
              }
              __syncwarp();
              ++num_gone;
              left -= static_cast<double>(w);
            }
          }
          next = base + at + 1;
          if (ok) {
            node = base + at;
            if (lane == 0) sh.path[length] = node;
            ++length;
            walk_c = 0.f;
            sum = 1.f;
            left = 1.0;
            num_gone = 0;
          }
        }
      }
      if (lane == 0) {
        sh.node = node;
        sh.length = length;
        sh.num_gone = num_gone;
        sh.c = walk_c;
        sh.todo = todo;
      }
    }
    __syncthreads();
    const int todo = sh.todo;
    c = sh.c;
    p_row = prm.target_probs + (static_cast<int64_t>(q_begin) + sh.node) * prm.target_stride;
    q_row = c > 0.f ? prm.draft_probs + (static_cast<int64_t>(q_begin) + sh.node) * prm.draft_stride : nullptr;
    all = row_sum(buffer);
    if (todo == 1) break;
    buffer ^= 1;
    sum = static_cast<float>(all) * (1.f / kUnits);
    __syncthreads();
  }
  if (all == 0 && (c > 0.f || sh.num_gone > 0)) {
    // nothing is left of the row (a rejection that rounding alone allows): the row itself
    __syncthreads();
    if (tid == 0) sh.num_gone = 0;
    __syncthreads();
    c = 0.f;
    q_row = nullptr;
    buffer ^= 1;
    all = row_sum(buffer);
  }

  // ----- the results ---------------------------------------------------------------------------
  if (rank == 0) {
    const int length = sh.length;
    for (int i = tid; i < prm.max_q_len; i += kThreads) kept[i] = i < length ? begin + sh.path[i] : -1;
    if (tid == 0) {
      prm.counts[b] = length;
      if (prm.begin != nullptr) prm.begin[b] = begin;
      if (all == 0) {
        prm.next_tokens[b] = -1;
        record_error(prm.err, kErrNoProbability);
      }
    }
  }
  if (all == 0) return;
  // the drawn number: floor(u T), and whose piece it falls into
  const double at = floor(static_cast<double>(prm.final_uniforms[b]) * static_cast<double>(all));
  unsigned long long t = at > 0.0 ? static_cast<unsigned long long>(at) : 0ull;  // (NaN: 0)
  if (t > all - 1) t = all - 1;
  for (int r = 0; r < rank; ++r) {
    if (t < sh.block_sum[buffer][r]) return;
    t -= sh.block_sum[buffer][r];
  }
  if (t >= sh.block_sum[buffer][rank]) return;
  for (int w = 0; w < warp; ++w) {
    if (t < sh.warp_sum[w]) return;
    t -= sh.warp_sum[w];
  }
  if (t >= sh.warp_sum[warp]) return;
  int x0 = from, batch = 0;
  while (t >= sh.batch_sum[warp][batch]) {
    t -= sh.batch_sum[warp][batch++];
    x0 += kDeep * 128;
  }
  float p[kDeep][4], q[kDeep][4];
  load_batch(x0, p, q);
  for (int i = 0; i < sh.num_gone; ++i) {
    const long long at = sh.gone[i] - x0;
    if (at < 0 || at >= kDeep * 128) continue;  // (the whole warp)
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[d][j] = at == d * 128 + lane * 4 + j ? 0.f : p[d][j];
  }
#pragma unroll
  for (int d = 0; d < kDeep; ++d) {
    const int x = x0 + d * 128 + lane * 4;
    uint32_t hi[4], lo[4];
    weights(p[d], q[d], hi, lo);
    unsigned long long v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (static_cast<unsigned long long>(hi[j]) << 21) + lo[j];
    const unsigned long long mine = v[0] + v[1] + v[2] + v[3];
    unsigned long long upto = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const unsigned long long before = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += before;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, t < upto);
    if (past != 0) {
      if (lane == __ffs(past) - 1) {
        t -= upto - mine;
        int j = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (j == k && t >= v[k]) {
            t -= v[k];
            ++j;
          }
        prm.next_tokens[b] = x + j;
      }
      return;
    }
    t -= __shfl_sync(0xffffffffu, upto, 31);
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream, bool use_pdl) {
  auto aligned = [](const float* x, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && stride % 4 == 0;
  };
  // whole rows on 16-byte boundaries: four probabilities a load
  const bool vec = p.vocab % 4 == 0 && aligned(p.target_probs, p.target_stride) &&
                   (p.draft_probs == nullptr || aligned(p.draft_probs, p.draft_stride));
  return fail_at(launch_kernel(vec ? verify_kernel<true> : verify_kernel<false>,
                               dim3(kCluster, static_cast<unsigned>(p.bs)), dim3(kThreads), 0, stream, use_pdl, p),
                 "cudaLaunchKernelEx");
}

}  // namespace pa

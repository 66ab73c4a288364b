// Pages of the cache: copied, shared between forked requests, handed out, given back, and moved
// to the front of their pools.
//
// State.  req_to_token rows hold slots (page * page_size + row), the whole page's whenever a page
// is handed out; page_refs counts the rows that hold a page, 0 where it is free.  Pages are handed
// out lowest first, so equal states give equal tables.
//
// Shape.  One thread block plans: it ranks the free pages by a scan of page_refs (reading stops
// when enough are found) and leaves (source, destination) pairs.  A grid applies the plan: table
// rows, and the pages of every pool in tasks of 16 KiB.  A list of up to PagesPools::kMax pools travels
// in the kernel's arguments, so a fork or a compaction over all layers is two launches.
//
// Bound by memory for copies, every byte read and written once (2.1 GB of a compaction 335 us, 6.4
// TB/s); by two launches and the scan for a few pages (a fork of one request into four, 8.5 MB copied,
// 11 to 12 us in a graph with the free before it; a free that finds nothing 2.5), and by the scan's rounds
// where nearly everything is taken (4 rows extended by a page, with the free after it: of 4096 pages 7.9
// us, of 65536 20, of 2^20 217).
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kTaskBytes = kThreads * 16 * 4;

// Inclusive scans over the block of one number a thread.  (Two sets of warp sums in turn: one
// barrier a scan.)
template <int kThreads>
struct Scan {
  int sums[2][32];
  __device__ __forceinline__ int operator()(int v, int& turn, int& total) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += up;
    }
    int* mine = sums[turn];
    turn ^= 1;
    if (lane == 31) mine[warp] = v;
    __syncthreads();
    int w = lane < kWarps ? mine[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += up;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return v + (warp > 0 ? before : 0);
  }
};

// Holders of a thread's four pages from `base` on.
__device__ __forceinline__ int4 holders(const int32_t* refs, int64_t num_pages, int64_t base) {
  const int64_t at = base + threadIdx.x * 4;
  return make_int4(at < num_pages ? refs[at] : 1, at + 1 < num_pages ? refs[at + 1] : 1,
                   at + 2 < num_pages ? refs[at + 2] : 1, at + 3 < num_pages ? refs[at + 3] : 1);
}

// The lowest `want` free pages, in order, to `list`; returns how many there are (all threads).
// `first`: holders(.., 0), which the plans ask for before they read their entries; then each round's are
// on their way during the scan before it.
template <int kThreads>
__device__ int find_free(const int32_t* refs, int64_t num_pages, int want, int32_t* list, Scan<kThreads>& scan,
                         int& turn, int4 first) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < want; base += kThreads * 4) {
    const int64_t at = base + threadIdx.x * 4;
    const int r[4] = {first.x, first.y, first.z, first.w};
    first = holders(refs, num_pages, base + kThreads * 4);
    int free = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) free += r[j] == 0;
    int total;
    int rank = found + scan(free, turn, total) - free;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r[j] == 0) {
        if (rank < want) list[rank] = static_cast<int32_t>(at + j);
        ++rank;
      }
    found += total;
  }
  return min(found, want);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) { return (tokens + page_size - 1) / page_size; }

// Row index and token count of an entry, checked; -1 where it is refused.
__device__ __forceinline__ int64_t checked_row(const PagesParams& p, const int64_t* rows, int i, bool report) {
  const int64_t row = rows[i];
  if (row >= 0 && row < p.num_rows) return row;
  if (report) record_error(p.err, kErrPoolRowOutOfRange);
  return -1;
}
__device__ __forceinline__ int checked_length(const PagesParams& p, const int32_t* lens, int i, bool report) {
  const int n = lens[i];
  if (n >= 0 && n <= p.max_seq_pages * p.page_size) return n;
  if (report) record_error(p.err, kErrSeqLenOutOfRange);
  return -1;
}

// Threads of a plan: 256 start sooner, 1024 read more pages and entries at a time.  Compaction looks
// at every page twice, one a thread (4096 pages: 12.1 us with 256 threads, 7.6 us with 1024); the
// others stop at the pages that they need, four a thread.
bool small_plan(const PagesParams& p, int64_t pages_a_round) {
  return p.num_pages <= 4 * pages_a_round && p.count <= 1024;
}

// ---- plans --------------------------------------------------------------------------------------

// Forks: a free page for every child whose last page is partly filled.
template <int kPlan>
__global__ void __launch_bounds__(kPlan) plan_fork_kernel(const PagesParams p) {
  __shared__ Scan<kPlan> scan;
  int turn = 0;
  trigger_dependents();  // (what applies the plan waits for its end)
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int4 first = holders(p.page_refs, p.num_pages, 0);
  int want = 0;
  for (int base = 0; base < p.count; base += kPlan) {
    const int i = base + tid;
    int needs = 0;
    if (i < p.count) {
      const int64_t parent = checked_row(p, p.rows, i, true), child = checked_row(p, p.children, i, true);
      const int n = checked_length(p, p.lens, i, true);
      int32_t src = -1;
      if (parent >= 0 && child >= 0 && n >= 0 && n % p.page_size != 0) {
        const int32_t slot = p.req_to_token[parent * p.row_stride + n / p.page_size * p.page_size];
        if (slot < 0 || slot / p.page_size >= p.num_pages) {
          record_error(p.err, kErrPageOutOfRange);
        } else if (p.page_refs[slot / p.page_size] <= 0) {
          record_error(p.err, kErrPageRefs);
        } else {
          src = slot / p.page_size;
        }
      }
      needs = src >= 0;
      p.src_pages[i] = src;
      p.granted[i] = parent >= 0 && child >= 0 && n >= 0 ? n : 0;
    }
    int total;
    const int rank = want + scan(needs, turn, total) - needs;
    if (i < p.count) p.dst_pages[i] = needs ? rank : -1;
    want += total;
  }
  __syncthreads();
  const int found = find_free(p.page_refs, p.num_pages, want, p.list, scan, turn, first);
  __syncthreads();
  for (int i = tid; i < p.count; i += kPlan) {
    const int rank = p.dst_pages[i];
    if (rank < 0) {
      // a last page that could not be read, or that nobody holds: the child has what is before it
      if (p.granted[i] % p.page_size != 0) p.granted[i] -= p.granted[i] % p.page_size;
      continue;
    }
    const int page = rank < found ? p.list[rank] : -1;
    p.dst_pages[i] = page;
    if (page >= 0) {
      p.page_refs[page] = 1;
    } else {
      record_error(p.err, kErrOutOfPages);
      p.granted[i] -= p.granted[i] % p.page_size;
    }
  }
}

// Growth: free pages for the pages of every request between its old and its new length.
template <int kPlan>
__global__ void __launch_bounds__(kPlan) plan_extend_kernel(const PagesParams p) {
  __shared__ Scan<kPlan> scan;
  int turn = 0;
  trigger_dependents();  // (what applies the plan waits for its end)
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int4 first = holders(p.page_refs, p.num_pages, 0);
  int want = 0;
  for (int base = 0; base < p.count; base += kPlan) {
    const int i = base + tid;
    int needs = 0;
    if (i < p.count) {
      const int64_t row = checked_row(p, p.rows, i, true);
      const int old_n = checked_length(p, p.lens, i, true), new_n = checked_length(p, p.new_lens, i, true);
      if (row >= 0 && old_n >= 0 && new_n >= 0)
        needs = max(0, pages_of(new_n, p.page_size) - pages_of(old_n, p.page_size));
    }
    // (more than there are pages is more than enough: the sums stay within 31 bits)
    needs = static_cast<int>(min(static_cast<int64_t>(needs), p.num_pages));
    int total;
    const int rank = want + scan(needs, turn, total) - needs;
    if (i < p.count) p.src_pages[i] = rank;
    want = static_cast<int>(min(static_cast<int64_t>(want) + total, p.num_pages));
  }
  __syncthreads();
  const int found = find_free(p.page_refs, p.num_pages, want, p.list, scan, turn, first);
  __syncthreads();
  for (int r = tid; r < found; r += kPlan) p.page_refs[p.list[r]] = 1;
  for (int i = tid; i < p.count; i += kPlan) {
    const int64_t row = checked_row(p, p.rows, i, false);
    const int old_n = checked_length(p, p.lens, i, false), new_n = checked_length(p, p.new_lens, i, false);
    if (row < 0 || old_n < 0 || new_n < 0) {
      p.dst_pages[i] = 0;
      p.granted[i] = max(old_n, 0);
      continue;
    }
    const int needs = max(0, pages_of(new_n, p.page_size) - pages_of(old_n, p.page_size));
    const int got = max(0, min(needs, found - p.src_pages[i]));
    p.dst_pages[i] = got;
    if (got < needs) record_error(p.err, kErrOutOfPages);
    p.granted[i] = got < needs ? (pages_of(old_n, p.page_size) + got) * p.page_size : max(old_n, new_n);
  }
}

// Compaction: live pages at or past the number of live pages move to the free ones before it.
template <int kPlan>
__global__ void __launch_bounds__(kPlan) plan_compact_kernel(const PagesParams p) {
  __shared__ Scan<kPlan> scan;
  int turn = 0;
  trigger_dependents();  // (what applies the plan waits for its end)
  grid_dependency_wait();
  const int tid = threadIdx.x;
  int live = 0;
  for (int64_t i = tid; i < p.num_pages; i += kPlan) live += p.page_refs[i] > 0;
  int total;
  scan(live, turn, total);
  const int count = total;
  int moves = 0, holes = 0;
  for (int64_t base = 0; base < p.num_pages; base += kPlan) {
    const int64_t i = base + tid;
    const bool used = i < p.num_pages && p.page_refs[i] > 0;
    const int moved = used && i >= count, hole = i < p.num_pages && !used && i < count;
    if (i < p.num_pages) p.page_map[i] = used ? static_cast<int32_t>(i) : -1;
    // (below `count` there are holes, from there on moves: one scan ranks both)
    const int rank = scan(moved + hole, turn, total) - (moved + hole);
    const int mine_holes = base + kPlan <= count ? total : -1;
    if (mine_holes >= 0) {
      if (hole) p.dst_pages[holes + rank] = static_cast<int32_t>(i);
      holes += total;
    } else if (base >= count) {
      if (moved) p.src_pages[moves + rank] = static_cast<int32_t>(i);
      moves += total;
    } else {  // the stretch that holds the border
      int of_holes;
      const int at = scan(hole, turn, of_holes) - hole;
      if (hole) p.dst_pages[holes + at] = static_cast<int32_t>(i);
      if (moved) p.src_pages[moves + rank - of_holes] = static_cast<int32_t>(i);
      holes += of_holes;
      moves += total - of_holes;
    }
  }
  __syncthreads();
  for (int r = tid; r < moves; r += kPlan) {  // (as many holes as moves)
    const int src = p.src_pages[r], dst = p.dst_pages[r];
    p.page_map[src] = dst;
    p.page_refs[dst] = p.page_refs[src];
    p.page_refs[src] = 0;
  }
  if (tid == 0) {
    *p.num_moves = moves;
    *p.num_live = count;
  }
}

// ---- what a plan does -----------------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ void copy_words(const void* src, void* dst, int64_t bytes, int thread, int threads) {
  const T* s = static_cast<const T*>(src);
  T* d = static_cast<T*>(dst);
  const int words = static_cast<int>(bytes / sizeof(T));
  for (int i0 = thread; i0 < words; i0 += 4 * threads) {
    T w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * threads < words) w[u] = s[i0 + u * threads];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * threads < words) d[i0 + u * threads] = w[u];
  }
}

__device__ __forceinline__ void copy_bytes(const void* src, void* dst, int64_t bytes, int thread, int threads) {
  if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | static_cast<uintptr_t>(bytes)) & 15) == 0) {
    copy_words<uint4>(src, dst, bytes, thread, threads);
  } else {
    copy_words<uint32_t>(src, dst, bytes, thread, threads);
  }
}

// The pages of every pool: tasks of 16 KiB of a large pool's page, and one task a pair for all
// small pools (scales), a warp a pool.
__device__ void copy_pages(const PagesParams& p, const PagesPools& pools, int64_t count, int64_t first_task) {
  const int64_t tasks = count * pools.tasks;
  for (int64_t task = first_task; task < tasks; task += gridDim.x) {
    const int64_t pair = task / pools.tasks;
    const int64_t src = p.src_pages[pair], dst = p.dst_pages[pair];
    if (src < 0 || dst < 0) continue;
    if (src >= p.num_pages || dst >= p.num_dst_pages) {
      if (threadIdx.x == 0) record_error(p.err, kErrPageOutOfRange);
      continue;
    }
    const int t = static_cast<int>(task - pair * pools.tasks);
    int i = 0;  // the pool that holds task t
    for (int step = 64; step > 0; step >>= 1)
      if (i + step < pools.large && pools.first_task[i + step] <= t) i += step;
    if (pools.large > 0 && t < pools.first_task[pools.large]) {
      const PagesPools::Pool& pool = pools.pool[i];
      const int64_t from = static_cast<int64_t>(t - pools.first_task[i]) * kTaskBytes;
      copy_bytes(static_cast<const char*>(pool.src) + src * pool.bytes + from,
                 static_cast<char*>(pool.dst) + dst * pool.bytes + from,
                 min(static_cast<int64_t>(kTaskBytes), pool.bytes - from), threadIdx.x, kThreads);
    } else {
      for (int s = pools.large + (threadIdx.x >> 5); s < pools.num; s += kThreads / 32) {
        const PagesPools::Pool& pool = pools.pool[s];
        copy_bytes(static_cast<const char*>(pool.src) + src * pool.bytes,
                   static_cast<char*>(pool.dst) + dst * pool.bytes, pool.bytes, threadIdx.x & 31, 32);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) copy_kernel(const PagesParams p, const __grid_constant__ PagesPools pools) {
  grid_dependency_wait();
  copy_pages(p, pools, p.num_moves != nullptr ? *p.num_moves : p.count, blockIdx.x);
}

// A page's slots in a row, `page` in place of what was there.
__device__ __forceinline__ void write_slots(const PagesParams& p, int64_t row, int at, int page, int thread, int threads) {
  for (int r = thread; r < p.page_size; r += threads) {
    const int64_t pos = static_cast<int64_t>(at) * p.page_size + r;
    if (pos < p.row_stride) p.req_to_token[row * p.row_stride + pos] = page * p.page_size + r;
  }
}

// Tables of 32 pages of a row are a task, a warp taking every eighth.
constexpr int kTablePages = 32;

// One holder more of a page that somebody holds.  (Looked at first: counts only rise in this launch, so a
// page that nobody held when it began is refused to every child alike.)
__device__ __forceinline__ bool hold(int32_t* refs) {
  if (*static_cast<volatile int32_t*>(refs) <= 0) return false;
  atomicAdd(refs, 1);
  return true;
}

// Forks: the child's row up to its last full page is the parent's, each of those pages has one
// holder more (a page that cannot be shared leaves -1); then the copied page's slots.
__global__ void __launch_bounds__(kThreads) apply_fork_kernel(const PagesParams p, const __grid_constant__ PagesPools pools) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int spans = (p.max_seq_pages + kTablePages - 1) / kTablePages;
  const int64_t tables = static_cast<int64_t>(p.count) * spans;
  int64_t task = blockIdx.x;
  for (; task < tables; task += gridDim.x) {
    const int i = static_cast<int>(task / spans);
    const int n = p.granted[i];
    if (n <= 0) continue;
    const int64_t parent = p.rows[i], child = p.children[i];
    const int first = static_cast<int>(task - static_cast<int64_t>(i) * spans) * kTablePages;
    for (int at = first + warp; at < min(first + kTablePages, pages_of(n, p.page_size)); at += kThreads / 32) {
      if (at == n / p.page_size) {
        write_slots(p, child, at, p.dst_pages[i], lane, 32);
        continue;
      }
      const int64_t pos = static_cast<int64_t>(at) * p.page_size;
      const int32_t* from = p.req_to_token + parent * p.row_stride + pos;
      int32_t* to = p.req_to_token + child * p.row_stride + pos;
      const int32_t slot = from[0];
      const bool known = slot >= 0 && slot / p.page_size < p.num_pages;
      for (int r = lane; r < p.page_size && pos + r < p.row_stride; r += 32) to[r] = from[r];
      bool shared = true;
      if (lane == 0) {
        shared = known && hold(&p.page_refs[slot / p.page_size]);
        if (!shared) record_error(p.err, known ? kErrPageRefs : kErrPageOutOfRange);
      }
      if (__any_sync(0xffffffffu, !shared))  // (the row first: nothing waits for the count where all is well)
        for (int r = lane; r < p.page_size && pos + r < p.row_stride; r += 32) to[r] = -1;
    }
  }
  copy_pages(p, pools, p.count, task - tables);
}

__global__ void __launch_bounds__(kThreads) apply_extend_kernel(const PagesParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int spans = (p.max_seq_pages + kTablePages - 1) / kTablePages;
  const int64_t tables = static_cast<int64_t>(p.count) * spans;
  for (int64_t task = blockIdx.x; task < tables; task += gridDim.x) {
    const int i = static_cast<int>(task / spans);
    const int got = p.dst_pages[i];
    const int first = static_cast<int>(task - static_cast<int64_t>(i) * spans) * kTablePages;
    if (first >= got) continue;
    const int begin = pages_of(p.lens[i], p.page_size);
    for (int k = first + warp; k < min(first + kTablePages, got); k += kThreads / 32)
      write_slots(p, p.rows[i], begin + k, p.list[p.src_pages[i] + k], lane, 32);
  }
}

__global__ void __launch_bounds__(kThreads) free_kernel(const PagesParams p) {
  grid_dependency_wait();
  const int64_t total = static_cast<int64_t>(p.count) * p.max_seq_pages;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < total;
       t += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int i = static_cast<int>(t / p.max_seq_pages), at = static_cast<int>(t - static_cast<int64_t>(i) * p.max_seq_pages);
    const int64_t row = checked_row(p, p.rows, i, at == 0);
    const int n = checked_length(p, p.lens, i, at == 0);
    const int keep = p.new_lens != nullptr ? checked_length(p, p.new_lens, i, at == 0) : 0;
    if (row < 0 || n < 0 || keep < 0 || at < pages_of(keep, p.page_size) || at >= pages_of(n, p.page_size)) continue;
    // (the exchange: a page that two entries of the list name is given back once)
    const int32_t slot = atomicExch(&p.req_to_token[row * p.row_stride + static_cast<int64_t>(at) * p.page_size], -1);
    if (slot < 0) continue;
    if (slot / p.page_size >= p.num_pages) {
      record_error(p.err, kErrPageOutOfRange);
    } else if (atomicSub(&p.page_refs[slot / p.page_size], 1) <= 0) {
      atomicAdd(&p.page_refs[slot / p.page_size], 1);
      record_error(p.err, kErrPageRefs);
    }
  }
}

__global__ void __launch_bounds__(kThreads) apply_compact_kernel(const PagesParams p, const __grid_constant__ PagesPools pools) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int spans = (p.max_seq_pages + kTablePages - 1) / kTablePages;
  const int64_t tables = static_cast<int64_t>(p.count) * spans;
  int64_t task = blockIdx.x;
  for (; task < tables; task += gridDim.x) {
    const int i = static_cast<int>(task / spans);
    const int first = static_cast<int>(task - static_cast<int64_t>(i) * spans) * kTablePages;
    const int64_t row = checked_row(p, p.rows, i, first == 0 && threadIdx.x == 0);
    const int n = checked_length(p, p.lens, i, first == 0 && threadIdx.x == 0);
    if (row < 0 || n < 0) continue;
    for (int at = first + warp; at < min(first + kTablePages, pages_of(n, p.page_size)); at += kThreads / 32) {
      const int32_t slot = p.req_to_token[row * p.row_stride + static_cast<int64_t>(at) * p.page_size];
      if (slot < 0) continue;
      if (slot / p.page_size >= p.num_pages) {
        if (lane == 0) record_error(p.err, kErrPageOutOfRange);
        continue;
      }
      const int page = p.page_map[slot / p.page_size];
      __syncwarp();
      // (a row that is listed twice may have been done already: its pages were free, -1)
      if (page >= 0 && page != slot / p.page_size) write_slots(p, row, at, page, lane, 32);
    }
  }
  copy_pages(p, pools, *p.num_moves, task - tables);
}

unsigned blocks_for(int64_t tasks) {
  // up to eight blocks an SM: 128 KiB in flight on each
  const int64_t most = 152 * 8;
  return static_cast<unsigned>(tasks < 1 ? 1 : tasks < most ? tasks : most);
}

// Pools [from, from + PagesPools::kMax) as kernel arguments, the large ones first.
PagesPools pack(const pa_page_pool* src, const pa_page_pool* dst, int32_t from, int32_t num) {
  PagesPools out = {};
  for (int pass = 0; pass < 2; ++pass) {
    for (int32_t i = from; i < num && i < from + PagesPools::kMax; ++i) {
      const bool large = src[i].page_bytes > 4096;
      if (large != (pass == 0)) continue;
      if (large) {
        out.first_task[out.large++] = out.tasks;
        out.tasks += static_cast<int32_t>((src[i].page_bytes + kTaskBytes - 1) / kTaskBytes);
      }
      out.pool[out.num++] = {src[i].base, dst[i].base, src[i].page_bytes};
    }
    if (pass == 0) out.first_task[out.large] = out.tasks;
  }
  if (out.num > out.large) ++out.tasks;
  return out;
}

}  // namespace

cudaError_t launch_pages_copy(const PagesParams& p, const pa_page_pool* src, const pa_page_pool* dst,
                              int32_t from, int32_t num, int64_t most, cudaStream_t stream, bool use_pdl) {
  for (; from < num; from += PagesPools::kMax) {
    const PagesPools pools = pack(src, dst, from, num);
    const cudaError_t e = launch_kernel(copy_kernel, dim3(blocks_for(most * pools.tasks)), dim3(kThreads), 0,
                                        stream, use_pdl, p, pools);
    if (e != cudaSuccess) return fail_at(e, "cudaLaunchKernelEx (copy)");
  }
  return cudaSuccess;
}

cudaError_t launch_pages_fork(const PagesParams& p, const pa_page_pool* pools, int32_t num,
                              cudaStream_t stream, bool use_pdl) {
  const bool small = small_plan(p, 1024);
  cudaError_t e = launch_kernel(small ? plan_fork_kernel<256> : plan_fork_kernel<1024>, dim3(1),
                                dim3(small ? 256 : 1024), 0, stream, use_pdl, p);
  if (e != cudaSuccess) return fail_at(e, "cudaLaunchKernelEx (plan)");
  const PagesPools first = pack(pools, pools, 0, num);
  const int64_t tables = static_cast<int64_t>(p.count) * ((p.max_seq_pages + kTablePages - 1) / kTablePages);
  e = launch_kernel(apply_fork_kernel, dim3(blocks_for(tables + static_cast<int64_t>(p.count) * first.tasks)),
                    dim3(kThreads), 0, stream, use_pdl, p, first);
  if (e != cudaSuccess) return fail_at(e, "cudaLaunchKernelEx (fork)");
  return launch_pages_copy(p, pools, pools, PagesPools::kMax, num, p.count, stream, use_pdl);
}

cudaError_t launch_pages_extend(const PagesParams& p, cudaStream_t stream, bool use_pdl) {
  const bool small = small_plan(p, 1024);
  cudaError_t e = launch_kernel(small ? plan_extend_kernel<256> : plan_extend_kernel<1024>, dim3(1),
                                dim3(small ? 256 : 1024), 0, stream, use_pdl, p);
  if (e != cudaSuccess) return fail_at(e, "cudaLaunchKernelEx (plan)");
  const int64_t tables = static_cast<int64_t>(p.count) * ((p.max_seq_pages + kTablePages - 1) / kTablePages);
  return fail_at(launch_kernel(apply_extend_kernel, dim3(blocks_for(tables)), dim3(kThreads), 0, stream, use_pdl, p),
                 "cudaLaunchKernelEx (extend)");
}

cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t stream, bool use_pdl) {
  const int64_t total = static_cast<int64_t>(p.count) * p.max_seq_pages;
  return fail_at(launch_kernel(free_kernel, dim3(blocks_for((total + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                               stream, use_pdl, p),
                 "cudaLaunchKernelEx (free)");
}

cudaError_t launch_pages_compact(const PagesParams& p, const pa_page_pool* pools, int32_t num,
                                 cudaStream_t stream, bool use_pdl) {
  const bool small = small_plan(p, 256);
  cudaError_t e = launch_kernel(small ? plan_compact_kernel<256> : plan_compact_kernel<1024>, dim3(1),
                                dim3(small ? 256 : 1024), 0, stream, use_pdl, p);
  if (e != cudaSuccess) return fail_at(e, "cudaLaunchKernelEx (plan)");
  const PagesPools first = pack(pools, pools, 0, num);
  const int64_t tables = static_cast<int64_t>(p.count) * ((p.max_seq_pages + kTablePages - 1) / kTablePages);
  e = launch_kernel(apply_compact_kernel, dim3(blocks_for(tables + p.num_pages / 2 * first.tasks)), dim3(kThreads),
                    0, stream, use_pdl, p, first);
  if (e != cudaSuccess) return fail_at(e, "cudaLaunchKernelEx (compact)");
  return launch_pages_copy(p, pools, pools, PagesPools::kMax, num, p.num_pages / 2, stream, use_pdl);
}

}  // namespace pa

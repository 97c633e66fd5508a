// Pages of the paged key/value cache: reserving, sharing (fork), freeing,
// copying and compacting them, with all state on the device, so that a step
// needs no host round trip and can be captured into a graph.
//
// State: refs[p] = how many sequences hold page p (0: free); a sequence's
// table row lists its pages in key order; only a page that is full is ever
// held by more than one sequence (a fork copies the last, partly filled one).
//
// Every call decides first and moves afterwards.  The decision is made by one
// block of 1024 threads (`plan`): it checks the call, finds the lowest free
// pages in index order (so results do not depend on thread order) and writes
// a list of page copies to the workspace, or refuses and writes an empty one.
// One block is enough because the decision is small next to a launch: it
// reads refs 16 pages a thread at a time and stops when it has enough (64K
// pages: 4 rounds).  The copies then run as a launch of their own over every
// pool, bound by memory (each byte read and written once).
#include "pages.cuh"

#include "common.cuh"

namespace ssattn {
namespace {

constexpr int kPlan = 1024;       // threads of a planning block
constexpr int kPerThread = 16;    // pages a planning thread looks at per round
constexpr int kCopy = 256;        // threads of a copying block
constexpr int kCopyUnroll = 8;    // 16-byte words a copying thread has in flight
constexpr int kCopyBytes = kCopy * kCopyUnroll * 16;  // 32 KB per block
constexpr int kSMs = 152;

// Workspace, in 32-bit words.
struct Plan {
  int32_t* head;   // [8]: 0 copies / movers, 1 accepted, 2 live pages
  int32_t* base;   // [n] first of an entry's pages in `list` (fork: its copy's target)
  int32_t* from;   // [n] source page of an entry's copy, -1: none
  int32_t* list;   // [num_pages] free pages found (compaction: holes)
  int32_t* map;    // [num_pages] compaction: movers' numbers by page
  int32_t* moved;  // [num_pages] compaction: movers
  uint32_t* bits;  // two sets of max(num_pages, num_rows) bits
};

__host__ __device__ long bit_words(int num_pages, int num_rows) {
  return (static_cast<long>(num_pages > num_rows ? num_pages : num_rows) + 31) / 32;
}

Plan plan_of(void* ws, int num_pages, int num_rows, int n) {
  Plan p;
  p.head = static_cast<int32_t*>(ws);
  p.base = p.head + 8;
  p.from = p.base + n;
  p.list = p.from + n;
  p.map = p.list + num_pages;
  p.moved = p.map + num_pages;
  p.bits = reinterpret_cast<uint32_t*>(p.moved + num_pages);
  return p;
}

__device__ __forceinline__ int tiles_of(int len) { return len <= 0 ? 0 : (len - 1) / kTile + 1; }

// Exclusive prefix sum over the block's threads; `total` receives the sum.
template <typename T>
__device__ T block_scan(T v, T* total) {
  __shared__ T warps[kPlan / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous scan's totals have been read
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warps[lane] = w;
  }
  __syncthreads();
  *total = warps[kPlan / 32 - 1];
  return x - v + (warp > 0 ? warps[warp - 1] : 0);
}

// Bit k: page first + k of this thread's kPerThread pages is in use (pages
// past the end count as `past`).
__device__ __forceinline__ uint32_t live_bits(const int32_t* refs, int num_pages, long first,
                                              uint32_t past) {
  uint32_t live = 0;
  if (first + kPerThread <= num_pages) {
#pragma unroll
    for (int q = 0; q < kPerThread / 4; ++q) {
      const int4 r = *reinterpret_cast<const int4*>(refs + first + 4 * q);
      live |= ((r.x > 0 ? 1u : 0u) | (r.y > 0 ? 2u : 0u) | (r.z > 0 ? 4u : 0u) | (r.w > 0 ? 8u : 0u))
              << (4 * q);
    }
  } else {
    for (int k = 0; k < kPerThread; ++k)
      live |= (first + k < num_pages ? (refs[first + k] > 0 ? 1u : 0u) : past) << k;
  }
  return live;
}

// The `need` lowest free pages, in order, into list; returns how many there are (up to need).
__device__ int find_free(const int32_t* refs, int num_pages, int need, int32_t* list) {
  int found = 0;
  for (long p0 = 0; p0 < num_pages && found < need; p0 += static_cast<long>(kPlan) * kPerThread) {
    const long first = p0 + static_cast<long>(threadIdx.x) * kPerThread;
    const uint32_t free_bits = ~live_bits(refs, num_pages, first, 1u) & ((1u << kPerThread) - 1);
    int total;
    int at = found + block_scan(__popc(free_bits), &total);
    for (uint32_t m = free_bits; m != 0 && at < need; m &= m - 1, ++at)
      list[at] = static_cast<int32_t>(first + __ffs(m) - 1);
    found += total;
  }
  return found < need ? found : need;
}

__device__ __forceinline__ bool set_bit(uint32_t* bits, int i) {  // true: it was set already
  return (atomicOr(&bits[i >> 5], 1u << (i & 31)) >> (i & 31)) & 1u;
}
__device__ __forceinline__ bool has_bit(const uint32_t* bits, int i) {
  return (*const_cast<const volatile uint32_t*>(&bits[i >> 5]) >> (i & 31)) & 1u;
}

// Clears both bit sets, marks `src` (nullable) in the first and `dst` in the
// second; true if an index is out of range, `dst` has one twice, or one of
// `dst` is also in `src` (a page or row copied over itself too).
__device__ bool bad_indices(uint32_t* bits, long words, const int32_t* src, const int32_t* dst, int n,
                            int limit) {
  for (long w = threadIdx.x; w < 2 * words; w += kPlan) bits[w] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int d = dst[i], s = src != nullptr ? src[i] : 0;
    if (d < 0 || d >= limit || s < 0 || s >= limit) {
      bad = true;
      continue;
    }
    if (src != nullptr) set_bit(bits, s);
    if (set_bit(bits + words, d)) bad = true;
  }
  __threadfence_block();
  if (__syncthreads_or(bad)) return true;
  if (src != nullptr)
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (has_bit(bits, dst[i])) bad = true;
  return __syncthreads_or(bad);
}

// ------------------------------------------------------------------ reserve
// Entry i: row rows[i] (or i) grows by add[i] keys.  All entries or none.
__global__ void __launch_bounds__(kPlan)
    reserve_kernel(const PageState s, const int32_t* rows, const int32_t* add, int n, int32_t* result,
                   Plan plan) {
  bool bad = false;
  if (rows != nullptr)
    bad = bad_indices(plan.bits, bit_words(s.num_pages, s.num_rows), nullptr, rows, n, s.num_rows);
  long need = 0;
  if (!bad) {
    for (int i0 = 0; i0 < n; i0 += kPlan) {
      const int i = i0 + threadIdx.x;
      long want = 0;
      if (i < n) {
        const int len = s.lens[rows != nullptr ? rows[i] : i];
        const long now = static_cast<long>(len) + add[i];
        if (len < 0 || add[i] < 0 || now > static_cast<long>(s.max_pages) * kTile)
          bad = true;
        else
          want = tiles_of(static_cast<int>(now)) - tiles_of(len);
      }
      long total;
      const long at = block_scan(want, &total);
      if (i < n) plan.base[i] = static_cast<int>(need + at);  // (used where need <= num_pages)
      need += total;
    }
    bad = __syncthreads_or(bad);
  }
  if (bad) {
    if (threadIdx.x == 0 && result != nullptr) *result = -1;
    return;
  }
  const int wanted = static_cast<int>(min(need, static_cast<long>(s.num_pages)));
  const int found = find_free(s.refs, s.num_pages, wanted, plan.list);
  if (threadIdx.x == 0 && result != nullptr)
    *result = static_cast<int>(min(need - found, 0x7fffffffL));
  if (found < need) return;
  __syncthreads();  // list and base
  for (int i = threadIdx.x >> 5; i < n; i += kPlan / 32) {  // a warp per entry
    const int row = rows != nullptr ? rows[i] : i;
    const int len = s.lens[row], now = len + add[i];
    const int t0 = tiles_of(len), t1 = tiles_of(now);
    for (int j = t0 + (threadIdx.x & 31); j < t1; j += 32) {
      const int p = plan.list[plan.base[i] + j - t0];
      s.table[static_cast<long>(row) * s.max_pages + j] = p;
      s.refs[p] = 1;
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) s.lens[row] = now;
  }
}

// --------------------------------------------------------------------- free
// One block per listed row; the block that takes a row's length frees it, so
// a row listed twice is freed once.
__global__ void __launch_bounds__(128) free_kernel(const PageState s, const int32_t* rows, int n) {
  __shared__ int length;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int row = rows[i];
    if (row < 0 || row >= s.num_rows) continue;
    __syncthreads();  // the previous entry's length has been read
    if (threadIdx.x == 0) length = atomicExch(&s.lens[row], 0);
    __syncthreads();
    const int tiles = min(tiles_of(length), s.max_pages);
    int32_t* t = s.table + static_cast<long>(row) * s.max_pages;
    for (int j = threadIdx.x; j < tiles; j += 128) {
      const int p = t[j];
      if (p >= 0 && p < s.num_pages) atomicSub(&s.refs[p], 1);
      t[j] = -1;
    }
  }
}

// ------------------------------------------------------------------- copies
// Bytes [c * kCopyBytes, ...) of page `from` over page `to` of one pool.
__device__ __forceinline__ void copy_chunk(unsigned char* pool, size_t page_bytes, int from, int to,
                                           long c) {
  const size_t at = static_cast<size_t>(c) * kCopyBytes;
  const uint4* src = reinterpret_cast<const uint4*>(pool + from * page_bytes + at);
  uint4* dst = reinterpret_cast<uint4*>(pool + to * page_bytes + at);
  const int words = static_cast<int>(min(static_cast<size_t>(kCopyBytes), page_bytes - at) / 16);
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int w = u * kCopy + threadIdx.x;
    if (w < words) v[u] = src[w];
  }
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int w = u * kCopy + threadIdx.x;
    if (w < words) dst[w] = v[u];
  }
}

// --------------------------------------------------------------------- fork
// Entry i: the empty row dst[i] becomes a second holder of row src[i]'s full
// pages, with a copy of its last page if that one is not full.
__global__ void __launch_bounds__(kPlan)
    fork_plan_kernel(const PageState s, const int32_t* src, const int32_t* dst, int n,
                     int32_t* result, Plan plan) {
  bool bad = bad_indices(plan.bits, bit_words(s.num_pages, s.num_rows), src, dst, n, s.num_rows);
  int need = 0;
  if (!bad) {
    for (int i0 = 0; i0 < n; i0 += kPlan) {
      const int i = i0 + threadIdx.x;
      int want = 0;
      if (i < n) {
        const int len = s.lens[src[i]];
        if (len < 0 || tiles_of(len) > s.max_pages || s.lens[dst[i]] != 0) bad = true;
        want = len > 0 && len % kTile != 0;
      }
      int total;
      const int at = block_scan(want, &total);
      if (i < n) plan.base[i] = want ? need + at : -1;
      need += total;
    }
    bad = __syncthreads_or(bad);
  }
  int found = 0;
  if (!bad) found = find_free(s.refs, s.num_pages, min(need, s.num_pages), plan.list);
  const bool accepted = !bad && found == need;
  if (threadIdx.x == 0) {
    plan.head[1] = accepted;
    if (result != nullptr) *result = bad ? -1 : need - found;
  }
  if (!accepted) return;
  __syncthreads();  // list and base
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int at = plan.base[i];
    int from = -1;
    if (at >= 0) {
      from = s.table[static_cast<long>(src[i]) * s.max_pages + s.lens[src[i]] / kTile];
      if (from < 0 || from >= s.num_pages) from = -1;  // (a table entry that names no page)
      plan.base[i] = plan.list[at];
    }
    plan.from[i] = from;
  }
}

// Blocks of entry i (of those from `entry0` on): one for its table row (with
// the first pools only), then one per (pool, chunk of a page).
__global__ void __launch_bounds__(kCopy)
    fork_apply_kernel(const PageState s, const int32_t* src, const int32_t* dst, Plan plan,
                      const PagePools pools, int chunks, int rows_too, int entry0) {
  if (plan.head[1] == 0) return;
  const int per = pools.count * chunks + rows_too, at = blockIdx.x / per;
  const int i = entry0 + at;
  int k = blockIdx.x - at * per;
  const int to = plan.base[i];
  if (rows_too && k-- == 0) {
    const int len = s.lens[src[i]], full = len / kTile;
    const int32_t* a = s.table + static_cast<long>(src[i]) * s.max_pages;
    int32_t* b = s.table + static_cast<long>(dst[i]) * s.max_pages;
    for (int j = threadIdx.x; j < s.max_pages; j += kCopy) {
      int p = -1;
      if (j < full) {
        p = a[j];
        if (p >= 0 && p < s.num_pages) atomicAdd(&s.refs[p], 1);
      } else if (j == full && to >= 0) {
        p = to;
        s.refs[p] = 1;
      }
      b[j] = p;
    }
    if (threadIdx.x == 0) s.lens[dst[i]] = len;
    return;
  }
  const int from = plan.from[i];
  if (from < 0) return;
  const int pool = k / chunks;
  copy_chunk(pools.base[pool], pools.page_bytes, from, to, k - pool * chunks);
}

// --------------------------------------------------------------------- copy
__global__ void __launch_bounds__(kPlan)
    copy_plan_kernel(int num_pages, const int32_t* src, const int32_t* dst, int n, int32_t* result,
                     Plan plan) {
  const bool bad = bad_indices(plan.bits, bit_words(num_pages, 0), src, dst, n, num_pages);
  if (threadIdx.x == 0) {
    plan.head[1] = !bad;
    if (result != nullptr) *result = bad ? -1 : 0;
  }
}

__global__ void __launch_bounds__(kCopy)
    copy_apply_kernel(const int32_t* src, const int32_t* dst, Plan plan, const PagePools pools,
                      int chunks, int entry0) {
  if (plan.head[1] == 0) return;
  const int per = pools.count * chunks, at = blockIdx.x / per;
  const int i = entry0 + at, k = blockIdx.x - at * per;
  const int pool = k / chunks;
  copy_chunk(pools.base[pool], pools.page_bytes, src[i], dst[i], k - pool * chunks);
}

// ------------------------------------------------------------------ compact
// With `live` pages in use, the ones at or above index `live` (as many as
// there are free ones below it) move down: the highest to the lowest free
// page, and so on.  Numbers: page p's among the movers counts from the top.
__global__ void __launch_bounds__(kPlan)
    compact_plan_kernel(const PageState s, int32_t* live_out, Plan plan) {
  constexpr long kRound = static_cast<long>(kPlan) * kPerThread;
  int live = 0;
  for (long p0 = 0; p0 < s.num_pages; p0 += kRound)
    live += __popc(live_bits(s.refs, s.num_pages, p0 + threadIdx.x * kPerThread, 0u));
  int all;
  block_scan(live, &all);
  int before0 = 0, holes = 0;
  for (long p0 = 0; p0 < s.num_pages; p0 += kRound) {
    const long first = p0 + threadIdx.x * kPerThread;
    const uint32_t bits = live_bits(s.refs, s.num_pages, first, 0u);
    int total;
    int before = before0 + block_scan(__popc(bits), &total);
    for (int k = 0; k < kPerThread && first + k < s.num_pages; ++k) {
      const int p = static_cast<int>(first + k);
      const bool used = (bits >> k) & 1u;
      if (p < all && !used) {
        plan.list[p - before] = p;
        ++holes;
      } else if (p >= all) {
        const int r = all - 1 - before;
        plan.map[p] = used ? r : -1;
        if (used) plan.moved[r] = p;
      }
      before += used;
    }
    before0 += total;
  }
  int movers;
  block_scan(holes, &movers);
  if (threadIdx.x == 0) {
    plan.head[0] = movers;
    plan.head[2] = all;
    if (live_out != nullptr) *live_out = all;
  }
}

// New reference counts and table (which may be the old ones: each thread
// reads an entry before it writes it, and a mover's count is moved by one
// thread), then the copies.
__global__ void __launch_bounds__(kCopy)
    compact_apply_kernel(const PageState s, int32_t* out_refs, int32_t* out_table, Plan plan,
                         const PagePools pools, int chunks, int state_too) {
  const int movers = plan.head[0], live = plan.head[2];
  const long stride = static_cast<long>(gridDim.x) * kCopy;
  const long t0 = static_cast<long>(blockIdx.x) * kCopy + threadIdx.x;
  if (state_too) {
    for (long p = t0; p < s.num_pages; p += stride) {
      const int r = s.refs[p];
      if (p < live) {
        if (r > 0) out_refs[p] = r;  // (a free one receives its mover's count)
      } else {
        if (r > 0) out_refs[plan.list[plan.map[p]]] = r;
        out_refs[p] = 0;
      }
    }
    const long entries = static_cast<long>(s.num_rows) * s.max_pages;
    for (long e = t0; e < entries; e += stride) {
      const int row = static_cast<int>(e / s.max_pages), j = static_cast<int>(e - static_cast<long>(row) * s.max_pages);
      int p = -1;
      if (j < tiles_of(s.lens[row])) {
        p = s.table[e];
        if (p >= live && p < s.num_pages) {
          const int r = plan.map[p];
          if (r >= 0 && r < movers) p = plan.list[r];
        }
      }
      out_table[e] = p;
    }
  }
  const long per = static_cast<long>(pools.count) * chunks, tasks = movers * per;
  for (long t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int i = static_cast<int>(t / per);
    const int k = static_cast<int>(t - i * per);
    const int pool = k / chunks;
    copy_chunk(pools.base[pool], pools.page_bytes, plan.moved[i], plan.list[i], k - pool * chunks);
  }
}

// Up to kMaxPools pools from `at` on.
PagePools some_pools(void* const* pools, int num_pools, int at, size_t page_bytes) {
  PagePools p{};
  p.page_bytes = page_bytes;
  p.count = num_pools - at < kMaxPools ? num_pools - at : kMaxPools;
  for (int i = 0; i < p.count; ++i) p.base[i] = static_cast<unsigned char*>(pools[at + i]);
  return p;
}

// Entries of `per` blocks each that one launch takes (a grid has 2^31 - 1 blocks; the plan has
// accepted all entries by then, so a longer list takes more launches).
int entries_of_a_launch(int per) { return 0x7fffffff / per; }

int chunks_of(size_t page_bytes) {
  return static_cast<int>((page_bytes + kCopyBytes - 1) / kCopyBytes);
}

}  // namespace

size_t pages_workspace(int num_pages, int num_rows, int n) {
  return 4 * (8 + 2 * static_cast<size_t>(n) + 3 * static_cast<size_t>(num_pages) +
              2 * static_cast<size_t>(bit_words(num_pages, num_rows)));
}

cudaError_t launch_pages_reserve(const PageState& s, const int32_t* rows, const int32_t* add, int n,
                                 int32_t* result, void* ws, cudaStream_t st) {
  reserve_kernel<<<1, kPlan, 0, st>>>(s, rows, add, n, result,
                                      plan_of(ws, s.num_pages, s.num_rows, n));
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageState& s, const int32_t* rows, int n, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  free_kernel<<<n < 16 * kSMs ? n : 16 * kSMs, 128, 0, st>>>(s, rows, n);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(void* const* pools, int num_pools, size_t page_bytes,
                              const PageState& s, const int32_t* src, const int32_t* dst, int n,
                              int32_t* result, void* ws, cudaStream_t st) {
  const Plan plan = plan_of(ws, s.num_pages, s.num_rows, n);
  fork_plan_kernel<<<1, kPlan, 0, st>>>(s, src, dst, n, result, plan);
  const int chunks = chunks_of(page_bytes);
  cudaError_t e = cudaGetLastError();
  for (int at = 0; e == cudaSuccess && n > 0 && (at == 0 || at < num_pools); at += kMaxPools) {
    const PagePools some = some_pools(pools, num_pools, at, page_bytes);
    const int per = some.count * chunks + (at == 0), most = entries_of_a_launch(per);
    for (int i = 0, m; e == cudaSuccess && i < n; i += m) {
      m = n - i < most ? n - i : most;
      fork_apply_kernel<<<static_cast<unsigned>(m) * per, kCopy, 0, st>>>(s, src, dst, plan, some, chunks,
                                                                          at == 0, i);
      e = cudaGetLastError();
    }
  }
  return e;
}

cudaError_t launch_pages_copy(void* const* pools, int num_pools, size_t page_bytes, int num_pages,
                              const int32_t* src, const int32_t* dst, int n, int32_t* result,
                              void* ws, cudaStream_t st) {
  const Plan plan = plan_of(ws, num_pages, 0, n);
  copy_plan_kernel<<<1, kPlan, 0, st>>>(num_pages, src, dst, n, result, plan);
  const int chunks = chunks_of(page_bytes);
  cudaError_t e = cudaGetLastError();
  for (int at = 0; e == cudaSuccess && n > 0 && at < num_pools; at += kMaxPools) {
    const PagePools some = some_pools(pools, num_pools, at, page_bytes);
    const int per = some.count * chunks, most = entries_of_a_launch(per);
    for (int i = 0, m; e == cudaSuccess && i < n; i += m) {
      m = n - i < most ? n - i : most;
      copy_apply_kernel<<<static_cast<unsigned>(m) * per, kCopy, 0, st>>>(src, dst, plan, some, chunks, i);
      e = cudaGetLastError();
    }
  }
  return e;
}

cudaError_t launch_pages_compact(void* const* pools, int num_pools, size_t page_bytes,
                                 const PageState& s, int32_t* out_refs, int32_t* out_table,
                                 int32_t* live, void* ws, cudaStream_t st) {
  const Plan plan = plan_of(ws, s.num_pages, s.num_rows, 0);
  compact_plan_kernel<<<1, kPlan, 0, st>>>(s, live, plan);
  cudaError_t e = cudaGetLastError();
  const int chunks = chunks_of(page_bytes);
  for (int at = 0; e == cudaSuccess && (at == 0 || at < num_pools); at += kMaxPools) {
    const PagePools some = some_pools(pools, num_pools, at, page_bytes);
    compact_apply_kernel<<<8 * kSMs, kCopy, 0, st>>>(s, out_refs, out_table, plan, some, chunks,
                                                     at == 0);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace ssattn

// What the planning blocks of the page calls share: prefix sums, the lowest free
// pages, checks of index lists, and the plan's place in the workspace.
#pragma once
#include "common.cuh"
#include "pages.cuh"

namespace ssattn {
namespace {

constexpr int kPlan = 1024;       // threads of a planning block
constexpr int kPerThread = 16;    // pages a planning thread looks at per round

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

[[maybe_unused]] Plan plan_of(void* ws, int num_pages, int num_rows, int n) {
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

}  // namespace
}  // namespace ssattn

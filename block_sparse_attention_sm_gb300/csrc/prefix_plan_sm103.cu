// What the sequences of a batch share: a tree over their page tables.
//
// Two sequences share a tile when their tables name the same pages up to it
// and both fill it (forked sequences, a prompt cached once).  Sorted by their
// rows of full pages, the sequences that share a stretch stand side by side,
// and with c[i] = number of tiles that places i - 1 and i have in common, each
// run of places between smaller values of c is a node of the tree: it holds the
// tiles from the larger of the two bounding values to its own.
//
// Two launches.  rank_kernel: block i compares row i with every other (a warp
// a pair, 32 pages a step; rows that differ in their first page, the usual
// case, end there): its place is the number of smaller rows, c its longest
// common stretch with one of them (the nearest smaller row has it).  tree_kernel:
// one thread a place looks left and right in shared memory for the run's ends.
// 64 rows of 256 pages that share 200: 6 us; most of it is latency.
#include "shared_decode.cuh"

namespace ssattn {
namespace {

constexpr int kRank = 512;
constexpr int kTree = 1024;

__device__ __forceinline__ int full_pages(int len, int max_pages) {
  return min(max(len, 0) / kTile, max_pages);
}

// (tiles that rows a and b share, whether b is the smaller); a whole warp.
__device__ __forceinline__ int common_pages(const int32_t* a, const int32_t* b, int n, int* diff) {
  const int lane = threadIdx.x & 31;
  for (int j = 0; j < n; j += 32) {
    const int x = j + lane < n ? a[j + lane] : 0, y = j + lane < n ? b[j + lane] : 0;
    // (an entry that names no page is shared with nobody)
    const uint32_t m = __ballot_sync(0xffffffffu, j + lane < n && (x != y || x < 0));
    if (m != 0) {
      const int at = __ffs(m) - 1;
      *diff = __shfl_sync(0xffffffffu, y < x ? -1 : y > x ? 1 : 0, at);
      return j + at;
    }
  }
  *diff = 0;
  return n;
}

__global__ void __launch_bounds__(kRank)
    rank_kernel(const int32_t* table, const int32_t* lens, int B, int max_pages, int32_t* plan) {
  __shared__ int smaller, longest;
  const int i = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) smaller = longest = 0;
  __syncthreads();
  const int32_t* mine = table + static_cast<long>(i) * max_pages;
  const int n_mine = full_pages(lens[i], max_pages);
  const int first = n_mine > 0 ? mine[0] : -1;
  int count = 0, most = 0;
  for (int j0 = warp * 32; j0 < B; j0 += kRank) {  // 32 rows: by their first page, a lane each
    const int j = j0 + lane;
    int n = 0, other = -1;
    if (j < B && j != i) {
      n = min(n_mine, full_pages(lens[j], max_pages));
      if (n > 0) other = table[static_cast<long>(j) * max_pages];
    }
    const bool open = j < B && j != i && n > 0 && other == first && first >= 0;
    bool less = false;
    if (j < B && j != i && !open) {
      const int nj = full_pages(lens[j], max_pages);
      if (n > 0 && other != first) less = other < first;
      else if (n > 0) less = j < i;  // (both name no page)
      else less = nj != n_mine ? nj < n_mine : j < i;
    }
    count += __popc(__ballot_sync(0xffffffffu, less));
    for (uint32_t m = __ballot_sync(0xffffffffu, open); m != 0; m &= m - 1) {
      const int at = __ffs(m) - 1, jj = j0 + at, nn = __shfl_sync(0xffffffffu, n, at);
      int diff;
      const int c = common_pages(mine, table + static_cast<long>(jj) * max_pages, nn, &diff);
      const int nj = full_pages(lens[jj], max_pages);
      const bool below = diff != 0 ? diff < 0 : c < nn ? jj < i : nj != n_mine ? nj < n_mine : jj < i;
      if (below) {
        ++count;
        most = max(most, c);
      }
    }
  }
  if (lane == 0) {
    atomicAdd(&smaller, count);
    atomicMax(&longest, most);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    plan[kPlanHead + smaller] = i;
    // c of that place, kept in its leaf until the tree is built
    plan[kPlanHead + B + smaller * kNodeWords + 2] = longest;
  }
}

__global__ void __launch_bounds__(kTree) tree_kernel(int B, int max_pages, int32_t* plan) {
  extern __shared__ int c[];  // [B + 1] common tiles of places i - 1 and i; c[0] = c[B] = 0
  int32_t* nodes = plan + kPlanHead + B;
  for (int i = threadIdx.x; i <= B; i += kTree) c[i] = i == 0 || i == B ? 0 : nodes[i * kNodeWords + 2];
  if (threadIdx.x < kPlanHead)
    plan[threadIdx.x] = threadIdx.x == 0 ? B : threadIdx.x == 1 ? max_pages : threadIdx.x == 2 ? kPlanMark : 0;
  __syncthreads();
  // The run of places around i - 1 and i that have c[i] tiles in common: its
  // name is the first i of it that has that value; its parent's is that of the
  // larger of the two values that bound it.
  auto run = [&](int i, int* lo, int* hi) {  // -> name; places [lo, hi)
    int name = i, l = i - 1, h = i + 1;
    while (c[l] >= c[i]) {  // (c[0] = 0 ends it)
      if (c[l] == c[i]) name = l;
      --l;
    }
    while (c[h] >= c[i]) ++h;
    *lo = l;
    *hi = h;
    return name;
  };
  auto bound = [&](int lo, int hi) { return c[lo] >= c[hi] ? lo : hi; };
  auto level = [&](int i) {  // 1: no node above it
    int n = 0;
    for (; c[i] > 0; ++n) {
      int lo, hi;
      run(i, &lo, &hi);
      i = bound(lo, hi);
    }
    return n;
  };
  auto name_of = [&](int i) {  // node of value c[i] around i, or -1
    if (c[i] == 0) return -1;
    int lo, hi;
    return B + run(i, &lo, &hi);
  };
  for (int i = threadIdx.x; i < B; i += kTree) {
    int first = 0, count = 0, t0 = 0, t1 = 0, parent = -1;
    if (i > 0 && c[i] > 0) {
      int lo, hi;
      if (run(i, &lo, &hi) == i && level(i) <= kPlanLevels) {
        const int up = bound(lo, hi);
        first = lo;
        count = hi - lo;
        t0 = c[up];
        t1 = c[i];
        parent = name_of(up);
      }
    }
    int32_t* n = nodes + (B + i) * kNodeWords;
    n[0] = first, n[1] = count, n[2] = t0, n[3] = t1, n[4] = parent;
    // The place's own tiles: those behind the deepest node above it that is kept.
    int up = bound(i, i + 1);
    for (int l = level(up); l > kPlanLevels; --l) {
      int lo, hi;
      run(up, &lo, &hi);
      up = bound(lo, hi);
    }
    n = nodes + i * kNodeWords;
    n[0] = i, n[1] = 1, n[2] = c[up], n[3] = -1, n[4] = name_of(up);
  }
}

}  // namespace

cudaError_t launch_prefix_plan(const int32_t* table, const int32_t* lens, int B, int max_pages,
                               int32_t* plan, cudaStream_t st) {
  rank_kernel<<<B, kRank, 0, st>>>(table, lens, B, max_pages, plan);
  tree_kernel<<<1, kTree, (B + 1) * sizeof(int), st>>>(B, max_pages, plan);
  return cudaGetLastError();
}

}  // namespace ssattn

// What the sequences of a batch share: a tree over their page tables.
//
// Two sequences share a tile when their tables name the same pages up to it
// and both fill it (forked sequences, a prompt cached once).  Sorted by their
// rows of full pages, the sequences that share a stretch stand side by side,
// and with c[i] = number of tiles that places i - 1 and i have in common, each
// run of places between smaller values of c is a node of the tree: it holds the
// tiles from the larger of the two bounding values to its own.
//
// Two launches.  rank_kernel: block i compares row i with every other, a warp a
// pair, 512 pages a step (rows that differ in their first page, the usual case,
// are sorted out before, a lane each): its place is the number of smaller rows, c
// its longest common stretch with one of them (the nearest smaller row has it).
// tree_kernel: a warp a place looks left and right for the run's ends, 32 places a
// step, in shared memory; then a thread a place goes up the tree.  Latency bounds both
// (48 places: 6.2 us and 3.2 us).  All pairs that begin on the same page are compared, so
// batches of one prefix cost their square: 64 places 11 us, 256 59 us, 1024 0.69 ms, 8192
// 42 ms (prefix of 256 pages).  A batch of up to 8 has both in one launch, the blocks of
// a cluster (8 places: 5.1 us against 4.3, but 3 us less of the host, which bounds such calls).
#include "launch.cuh"
#include "ptx_pair_sm103.cuh"
#include "shared_decode.cuh"

namespace ssattn {
namespace {

constexpr int kRank = 1024;
constexpr int kTree = 1024;
constexpr int kCluster = 8;  // blocks of a cluster
static_assert(kRank == kTree, "one block does both");
constexpr int kPlace = sizeof(int) + 2 * sizeof(uint16_t);  // shared memory of a place
static_assert(kPlanMaxB < 65536, "places in 16 bits");

__device__ __forceinline__ int full_pages(int len, int max_pages) {
  return min(max(len, 0) / kTile, max_pages);
}

// Tiles that rows a and b share, of n; *diff: how b compares with a behind them.  A whole warp.
__device__ __forceinline__ int common_pages(const int32_t* a, const int32_t* b, int n, int* diff) {
  constexpr int U = 16;  // words of each row that a lane has in flight
  const int lane = threadIdx.x & 31;
  for (int j0 = 0; j0 < n; j0 += 32 * U) {
    int x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + 32 * u + lane;
      x[u] = j < n ? a[j] : 0;
      y[u] = j < n ? b[j] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (an entry that names no page is shared with nobody)
      const uint32_t m = __ballot_sync(0xffffffffu, j0 + 32 * u + lane < n && (x[u] != y[u] || x[u] < 0));
      if (m != 0) {
        const int at = __ffs(m) - 1;
        *diff = __shfl_sync(0xffffffffu, y[u] < x[u] ? -1 : y[u] > x[u] ? 1 : 0, at);
        return j0 + 32 * u + at;
      }
    }
  }
  *diff = 0;
  return n;
}

// Row i: its place, and its longest common stretch with a smaller row.
__device__ __forceinline__ void rank_row(const int32_t* table, const int32_t* lens, int i, int B, int max_pages, int32_t* plan) {
  __shared__ int smaller, longest, n_open;
  __shared__ int open[kRank], open_n[kRank];  // rows that begin as row i does, and their full pages
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) smaller = longest = 0;
  const int32_t* mine = table + static_cast<long>(i) * max_pages;
  const int n_mine = full_pages(lens[i], max_pages);
  const int first = n_mine > 0 ? mine[0] : -1;
  int count = 0, most = 0;
  for (int j0 = 0; j0 < B; j0 += kRank) {
    __syncthreads();
    if (threadIdx.x == 0) n_open = 0;
    __syncthreads();
    const int j = j0 + threadIdx.x;
    if (j < B && j != i) {
      const int nj = full_pages(lens[j], max_pages), n = min(n_mine, nj);
      const int other = n > 0 ? table[static_cast<long>(j) * max_pages] : -1;
      if (n > 0 && other == first && first >= 0) {
        const int at = atomicAdd(&n_open, 1);
        open[at] = j;
        open_n[at] = nj;
      } else if (n > 0) {
        count += other != first ? other < first : j < i;  // (both name no page: by number)
      } else {
        count += nj != n_mine ? nj < n_mine : j < i;
      }
    }
    __syncthreads();
    for (int q = warp; q < n_open; q += kRank / 32) {
      const int jj = open[q], nj = open_n[q], n = min(n_mine, nj);
      int diff;
      const int c = common_pages(mine, table + static_cast<long>(jj) * max_pages, n, &diff);
      const bool below = diff != 0 ? diff < 0 : c < n ? jj < i : nj != n_mine ? nj < n_mine : jj < i;
      if (below) {
        count += lane == 0;
        most = max(most, c);
      }
    }
  }
  count = __reduce_add_sync(0xffffffffu, count);
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

// The tree from the ranks, by one block; `c`: kPlace bytes a place and one more.
__device__ __forceinline__ void build_tree(int B, int max_pages, int32_t* plan, int* c) {
  // c [B + 1]: common tiles of places i - 1 and i; c[0] = c[B] = 0
  auto* up = reinterpret_cast<uint16_t*>(c + B + 1);  // [B + 1] an i of the parent's run
  uint16_t* name = up + B + 1;                        // [B + 1] the run's name
  int32_t* nodes = plan + kPlanHead + B;
  for (int i = threadIdx.x; i <= B; i += kTree) c[i] = i == 0 || i == B ? 0 : __ldcg(&nodes[i * kNodeWords + 2]);
  if (threadIdx.x < kPlanHead)
    plan[threadIdx.x] = threadIdx.x == 0 ? B : threadIdx.x == 1 ? max_pages : threadIdx.x == 2 ? kPlanMark : 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  auto bound = [&](int lo, int hi) { return c[lo] >= c[hi] ? lo : hi; };  // the parent's value
  // The runs, a warp each: the places around i - 1 and i that have c[i] > 0 tiles in
  // common, [lo, hi).  A run's name is the first i of it that has that value.
  for (int i = threadIdx.x >> 5; i < B; i += kTree / 32) {
    int32_t* n = nodes + (B + i) * kNodeWords;
    const int v = c[i];
    int first = 0, count = 0, t0 = 0, t1 = 0;
    if (v > 0) {
      int at = i, l = i - 1, h = i + 1;
      while (true) {  // (c[0] = 0 ends it)
        const int x = l - lane >= 0 ? c[l - lane] : -1;
        const uint32_t stop = __ballot_sync(0xffffffffu, x < v), same = __ballot_sync(0xffffffffu, x == v);
        const uint32_t seen = stop != 0 ? same & ((1u << (__ffs(stop) - 1)) - 1) : same;
        if (seen != 0) at = l - (31 - __clz(seen));
        if (stop != 0) {
          l -= __ffs(stop) - 1;
          break;
        }
        l -= 32;
      }
      while (true) {  // (c[B] = 0)
        const uint32_t stop = __ballot_sync(0xffffffffu, (h + lane <= B ? c[h + lane] : -1) < v);
        if (stop != 0) {
          h += __ffs(stop) - 1;
          break;
        }
        h += 32;
      }
      if (at == i) first = l, count = h - l, t0 = c[bound(l, h)], t1 = v;
      if (lane == 0) {
        name[i] = static_cast<uint16_t>(at);
        up[i] = static_cast<uint16_t>(bound(l, h));
      }
    }
    if (lane == 0) n[0] = first, n[1] = count, n[2] = t0, n[3] = t1;
  }
  __syncthreads();
  // The nodes above each place, a thread each.
  auto level = [&](int i) {  // nodes from i's up
    int n = 0;
    for (; c[i] > 0; i = up[i]) ++n;
    return n;
  };
  int32_t* above = nodes + 2 * B * kNodeWords;
  for (int i = threadIdx.x; i < B; i += kTree) {
    if (level(i) > kPlanLevels) {  // (not kept)
      int32_t* n = nodes + (B + i) * kNodeWords;
      n[0] = n[1] = n[2] = n[3] = 0;
    }
    // From the deepest node that is kept up; the place's own tiles are those behind that one's.
    int at = bound(i, i + 1);
    for (int l = level(at); l > kPlanLevels; --l) at = up[at];
    int32_t* n = nodes + i * kNodeWords;
    n[0] = i, n[1] = 1, n[2] = c[at], n[3] = -1;
    for (int k = 0; k < kPlanLevels; ++k) {
      const bool some = c[at] > 0;
      above[i * kPlanLevels + k] = some ? B + name[at] : -1;
      if (some) at = up[at];
    }
  }
}

__global__ void __launch_bounds__(kRank)
    rank_kernel(const int32_t* table, const int32_t* lens, int B, int max_pages, int32_t* plan) {
  rank_row(table, lens, blockIdx.x, B, max_pages, plan);
}

__global__ void __launch_bounds__(kTree) tree_kernel(int B, int max_pages, int32_t* plan) {
  extern __shared__ int c[];
  let_next_start();
  wait_for_previous();
  build_tree(B, max_pages, plan, c);
}

// Both for a batch that a cluster holds.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kRank)
    small_plan_kernel(const int32_t* table, const int32_t* lens, int B, int max_pages, int32_t* plan) {
  __shared__ int c[((kCluster + 1) * kPlace + 3) / 4];
  let_next_start();
  if (blockIdx.x < B) rank_row(table, lens, blockIdx.x, B, max_pages, plan);
  __syncwarp();
  cluster_sync_all();  // (what the blocks have written to the plan as well)
  if (blockIdx.x == 0) build_tree(B, max_pages, plan, c);
}

}  // namespace

cudaError_t launch_prefix_plan(const int32_t* table, const int32_t* lens, int B, int max_pages,
                               int32_t* plan, cudaStream_t st) {
  if (B <= kCluster) {
    small_plan_kernel<<<kCluster, kRank, 0, st>>>(table, lens, B, max_pages, plan);
    return cudaGetLastError();
  }
  rank_kernel<<<B, kRank, 0, st>>>(table, lens, B, max_pages, plan);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(tree_kernel), (kPlanMaxB + 1) * kPlace, done);
  return e != cudaSuccess ? e : launch_behind(tree_kernel, 1, kTree, (B + 1) * kPlace, st, B, max_pages, plan);
}

}  // namespace ssattn

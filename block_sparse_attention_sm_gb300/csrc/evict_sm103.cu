// Eviction from the paged cache by accumulated attention weight: each listed
// sequence is cut back to `keep` keys, every KV head of every layer choosing
// its own (the newest `recent` of them, and of the older ones those of largest
// weight), in the pages themselves.
//
// choose_kernel: one block a (sequence, layer, head).  The keep - recent
// largest of L - recent fp32 weights by radix selection: three histograms (11,
// 11 and 10 bits of the weight as an unsigned number in the same order) give
// the smallest kept weight exactly, then one pass in the order of the keys
// takes what is above it and the first of those equal to it, and writes their
// places.  Up to 16384 keys the weights are read once and stay in registers (4 bytes a
// key next to the 4 d of keys and values that are moved); of longer sequences each of the passes
// reads them again, a block a list: 3 sequences of 64K 154 us, one of 200K 463.
// Block 0 of the first such launch decides, as the other page calls do: it
// checks the call, gives fresh pages to those that other sequences hold too
// (they are read, never written), and takes note of the old and new pages.
//
// move_kernel: kept rows move to the front of the sequence's pages.  Row d
// comes from src[d] >= d with src ascending, so a block that walks d upwards
// and has read the rows of a piece [d0, d1) before it writes it can move them in
// place: pieces behind read from src >= d1, which is not written yet.  A block
// has (sequence, head, pool) to itself, or 64-byte columns of it where
// there are few; it keeps kStages pieces in flight with asynchronous copies.
// The record of weights moves along, and the tables, lengths and counts follow.
//
// Bound by memory: kept rows are read and written once (16 sequences of 8K-12K keys cut to 4K
// in four layers, 2.2 GB: 433 us, 73% of the copy rate; rows of 256 bytes from scattered places).  Small
// calls are two launches: 4 sequences of 900, 6.7 and 6.1 us.
#include "evict.cuh"

#include "common.cuh"
#include "launch.cuh"
#include "pages_plan.cuh"
#include "ptx_sm103.cuh"

namespace ssattn {
namespace {

constexpr int kSMs = 152;
constexpr int kChoose = 1024;  // threads of a choosing block (kPlan: block 0 plans)
static_assert(kChoose == kPlan, "block 0 of a choosing launch plans");
constexpr int kBins = 2048;
constexpr int kMove = 256;
constexpr int kRounds = 2;                        // 16-byte words of a piece that a thread has
constexpr int kPieceBytes = kRounds * kMove * 16;  // rows that a moving block reads before it writes them
constexpr int kStages = 4;
constexpr int kGroup = 16;     // layers of a launch

struct Cut {      // what becomes of a listed sequence
  int row, len, now;
  int fresh;      // pages that others hold too are replaced
};

// Workspace.
struct Space {
  int32_t* head;   // [0]: accepted
  Cut* cut;        // [n]
  int32_t* base;   // [n] first of a sequence's fresh pages in `list`
  int32_t* entry;  // [num_rows] which listed sequence a row is, -1: none
  int32_t* list;   // [num_pages] lowest free pages
  int32_t* from;   // [n][max_pages] old pages
  int32_t* to;     // [n][max_pages] new pages
  uint32_t* bits;
  int32_t* src;    // [layers of a launch][n][Hkv][max_pages * 128] kept keys
};

constexpr size_t up16(size_t n) { return (n + 15) / 16 * 16; }

size_t space_of(Space* s, void* ws, int num_pages, int num_rows, int max_pages, int n, int Hkv, int layers) {
  char* base = static_cast<char*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* here = base + at;
    at += up16(bytes);
    return here;
  };
  const size_t N = n, W = max_pages;
  Space x;
  x.head = reinterpret_cast<int32_t*>(take(32));
  x.cut = reinterpret_cast<Cut*>(take(N * sizeof(Cut)));
  x.base = reinterpret_cast<int32_t*>(take(N * 4));
  x.entry = reinterpret_cast<int32_t*>(take(static_cast<size_t>(num_rows) * 4));
  x.list = reinterpret_cast<int32_t*>(take(static_cast<size_t>(num_pages) * 4));
  x.from = reinterpret_cast<int32_t*>(take(N * W * 4));
  x.to = reinterpret_cast<int32_t*>(take(N * W * 4));
  x.bits = reinterpret_cast<uint32_t*>(take(2 * static_cast<size_t>(bit_words(num_pages, num_rows)) * 4));
  x.src = reinterpret_cast<int32_t*>(take(static_cast<size_t>(layers) * N * Hkv * W * kTile * 4));
  if (s != nullptr) *s = x;
  return at;
}

int layers_of_a_launch(int num_layers, int per_layer) {
  const int fit = kMaxPools / per_layer < kGroup ? kMaxPools / per_layer : kGroup;
  return num_layers < fit ? num_layers : fit;
}

struct Layers {
  const float* weights[kGroup];
  float* out[kGroup];
  int count;
};

struct Call {
  PageState s;
  const int32_t* rows;
  const int32_t* keep;
  int n, recent, Hkv;
  int32_t* out_refs;
  int32_t* out_table;
  int32_t* out_lens;
  int32_t* result;
};

// ---------------------------------------------------------------------- plan
__device__ void plan_block(const Call& c, const Space& w) {
  const PageState& s = c.s;
  bool bad = c.rows != nullptr && bad_indices(w.bits, bit_words(s.num_pages, s.num_rows), nullptr, c.rows, c.n, s.num_rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!bad) {
    for (int i = threadIdx.x; i < c.n; i += kPlan) {
      const int row = c.rows != nullptr ? c.rows[i] : i;
      const int len = s.lens[row], keep = c.keep[i];
      if (len < 0 || len > s.max_pages * kTile || keep < 0) bad = true;
      w.cut[i] = Cut{row, len, min(len, keep), 0};
    }
    bad = __syncthreads_or(bad);
  }
  // pages that a cut sequence keeps and others hold too
  long need = 0;
  if (!bad) {
    for (int i = warp; i < c.n; i += kPlan / 32) {
      const Cut x = w.cut[i];
      int count = 0;
      if (x.now < x.len)
        for (int j = lane; j < tiles_of(x.now); j += 32) {
          const int p = s.table[static_cast<long>(x.row) * s.max_pages + j];
          count += p >= 0 && p < s.num_pages && s.refs[p] > 1;
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
      if (lane == 0) {
        w.base[i] = count;
        w.cut[i].fresh = count;
      }
    }
    __syncthreads();
    for (int i0 = 0; i0 < c.n; i0 += kPlan) {
      const int i = i0 + threadIdx.x;
      long total;
      const long at = block_scan(static_cast<long>(i < c.n ? w.base[i] : 0), &total);
      if (i < c.n) w.base[i] = static_cast<int>(need + at);
      need += total;
    }
  }
  int found = 0;
  if (!bad) found = find_free(s.refs, s.num_pages, static_cast<int>(min(need, static_cast<long>(s.num_pages))), w.list);
  const bool accepted = !bad && found >= need;
  if (threadIdx.x == 0) {
    w.head[0] = accepted;
    if (c.result != nullptr) *c.result = bad ? -1 : static_cast<int>(min(need - found, 0x7fffffffL));
  }
  if (!accepted) return;
  __syncthreads();  // base, list
  if (c.out_refs != s.refs)
    for (int p = threadIdx.x; p < s.num_pages; p += kPlan) c.out_refs[p] = s.refs[p];
  for (int r = threadIdx.x; r < s.num_rows; r += kPlan) w.entry[r] = -1;
  __syncthreads();
  // old and new pages, before any count changes
  for (int i = warp; i < c.n; i += kPlan / 32) {
    const Cut x = w.cut[i];
    if (lane == 0) w.entry[x.row] = i;
    const int old = tiles_of(x.len), now = tiles_of(x.now);
    int32_t* from = w.from + static_cast<long>(i) * s.max_pages;
    int32_t* to = w.to + static_cast<long>(i) * s.max_pages;
    int at = w.base[i];
    for (int j0 = 0; j0 < old; j0 += 32) {
      const int j = j0 + lane;
      const int p = j < old ? s.table[static_cast<long>(x.row) * s.max_pages + j] : -1;
      const bool shared = x.now < x.len && j < now && p >= 0 && p < s.num_pages && s.refs[p] > 1;
      const uint32_t m = __ballot_sync(0xffffffffu, shared);
      if (j < old) {
        from[j] = p;
        to[j] = j >= now ? -1 : shared ? w.list[at + __popc(m & ((1u << lane) - 1))] : p;
      }
      at += __popc(m);
    }
  }
  __syncthreads();
  // pages given up lose a holder, fresh ones have one
  for (int i = warp; i < c.n; i += kPlan / 32) {
    const Cut x = w.cut[i];
    for (int j = lane; j < tiles_of(x.len); j += 32) {
      const int p = w.from[static_cast<long>(i) * s.max_pages + j], q = w.to[static_cast<long>(i) * s.max_pages + j];
      if (p == q) continue;
      if (p >= 0 && p < s.num_pages) atomicSub(&c.out_refs[p], 1);
      if (q >= 0) c.out_refs[q] = 1;
    }
  }
}

// -------------------------------------------------------------------- choose
// A weight as an unsigned number of the same order; NaN below everything.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kChoose, 2)
    choose_kernel(const Call c, const Space w, const Layers layers, int plan_too) {
  let_next_start();
  if (plan_too && blockIdx.x == 0) {
    plan_block(c, w);
    return;
  }
  const int at = blockIdx.x - plan_too;
  const int h = at % c.Hkv, i = at / c.Hkv % c.n, layer = at / c.Hkv / c.n;
  const PageState& s = c.s;
  const int row = c.rows != nullptr ? c.rows[i] : i;
  if (row < 0 || row >= s.num_rows) return;
  const int len = max(0, min(s.lens[row], s.max_pages * kTile)), keep = max(0, c.keep[i]);
  if (len <= keep) return;
  const int newest = min(keep, c.recent), rest = len - newest, best = keep - newest;
  const long width = static_cast<long>(s.max_pages) * kTile;
  const float* weight = layers.weights[layer] + (static_cast<long>(row) * c.Hkv + h) * width;
  int32_t* src = w.src + ((static_cast<long>(layer) * c.n + i) * c.Hkv + h) * width;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // Each warp has a run of keys, whole words of 32 (a lane each).  Up to kHeld words
  // of it stay in registers; longer runs are read again, kHeld words at a time, in
  // each of the passes.
  constexpr int kHeld = 16;
  const int words = (len + 31) / 32, each = (words + kChoose / 32 - 1) / (kChoose / 32);
  const int w0 = min(words, warp * each), w1 = min(words, w0 + each);
  uint32_t u[kHeld];
  int held = -1;  // first word that is held
  auto hold = [&](int w) {
    if (held == w) return;
    held = w;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int k = (w + i) * 32 + lane;
      u[i] = w + i < w1 && k < rest ? order_of(weight[k]) : 0u;
    }
  };

  // The value of the best-th largest of weight[0, rest), and how many of those equal to it are kept.
  __shared__ int bins[kBins];
  __shared__ int s_bin, s_above;
  uint32_t value = 0;
  int wanted = best;
  if (best > 0 && best < rest) {
    int low = 32;  // bits of `value` from here up are known
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int width_bits = pass < 2 ? 11 : 10;
      const uint32_t known = pass == 0 ? 0u : 0xffffffffu << low;
      low -= width_bits;
      for (int b = tid; b < kBins; b += kChoose) bins[b] = 0;
      __syncthreads();
#pragma unroll 1
      for (int w = w0; w < w1; w += kHeld) {
        hold(w);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (w + i >= w1) break;
          // (what lies behind the older keys counts as 0, below which nothing is: the counts above a bin are right)
          const int bin = static_cast<int>((u[i] >> low) & ((1u << width_bits) - 1));
          if ((u[i] & known) == value) atomicAdd(&bins[bin], 1);  // (lanes that add one to the same word are counted by the hardware)
        }
      }
      __syncthreads();
      // from the top: thread t has bins 2047 - 2t and below it
      const int hi = bins[kBins - 1 - 2 * tid], lo = bins[kBins - 2 - 2 * tid];
      int total;
      const int above = block_scan(hi + lo, &total);
      if (above < wanted && above + hi >= wanted) {
        s_bin = kBins - 1 - 2 * tid;
        s_above = above;
      } else if (above + hi < wanted && above + hi + lo >= wanted) {
        s_bin = kBins - 2 - 2 * tid;
        s_above = above + hi;
      }
      __syncthreads();
      value |= static_cast<uint32_t>(s_bin) << low;
      wanted -= s_above;
    }
  }
  // wanted: of the weights equal to `value`; all of them if every older key is kept, none if none is.
  const bool all = best >= rest, none = best <= 0;
  auto above = [&](int k, uint32_t x) { return k < len && (k >= rest || all || (!none && x > value)); };
  auto equal = [&](int k, uint32_t x) { return k < rest && !all && !none && x == value; };
  int n_above = 0, n_equal = 0;  // of the warp's keys
#pragma unroll 1
  for (int w = w0; w < w1; w += kHeld) {
    hold(w);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (w + i >= w1) break;
      const int k = (w + i) * 32 + lane;
      n_above += __popc(__ballot_sync(0xffffffffu, w + i < w1 && above(k, u[i])));
      n_equal += __popc(__ballot_sync(0xffffffffu, w + i < w1 && equal(k, u[i])));
    }
  }
  int total;
  const int equal_before = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? n_equal : 0, &total), 0);
  const int taken = max(0, min(n_equal, wanted - equal_before));
  int out = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? n_above + taken : 0, &total), 0);
  int left = all || none ? 0 : taken;
#pragma unroll 1
  for (int w = w0; w < w1; w += kHeld) {
    hold(w);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (w + i >= w1) break;
      const int k = (w + i) * 32 + lane;
      const uint32_t e = __ballot_sync(0xffffffffu, w + i < w1 && equal(k, u[i]));
      const bool tie = ((e >> lane) & 1u) && __popc(e & ((1u << lane) - 1)) < left;
      left -= min(left, __popc(e));
      const uint32_t kept = __ballot_sync(0xffffffffu, tie || (w + i < w1 && above(k, u[i])));
      if ((kept >> lane) & 1u) {
        const int d = out + __popc(kept & ((1u << lane) - 1));
        if (d < keep) src[d] = k;
      }
      out += __popc(kept);
    }
  }
}

// ---------------------------------------------------------------------- move
__device__ __forceinline__ void copy_async16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows of one (sequence, head, pool), columns [column, column + 16 words).  A piece
// is kRounds rows a thread: what it copies in the piece after the next ones is looked
// up before it waits for this one.
__device__ void move_rows(const Call& c, const Space& w, unsigned char* pool, size_t page_bytes, int i, int h,
                          const int32_t* src, int row_bytes, int column, int words, unsigned char* stage) {
  const Cut x = w.cut[i];
  const int32_t* from = w.from + static_cast<long>(i) * c.s.max_pages;
  const int32_t* to = w.to + static_cast<long>(i) * c.s.max_pages;
  const int lead = threadIdx.x / words, word = threadIdx.x - lead * words;
  const int step = kMove / words, rows = kRounds * step;  // rows that the block takes at once, of a piece
  const bool busy = lead < step;
  unsigned char* mine = pool + static_cast<size_t>(h) * kTile * row_bytes + column + word * 16;
  const uint32_t place = smem_u32(stage) + (lead * words + word) * 16;  // in a stage, of the first row
  const int pieces = (x.now + rows - 1) / rows;
  auto valid = [&](int p) { return p >= 0 && p < c.s.num_pages; };
  // Pieces in front that stay where they are (src[d] - d never falls, so a piece whose
  // last row stays does so as a whole).
  int first = 0;
  if (x.fresh == 0) {
    for (int q0 = 0; q0 < pieces; q0 += kMove) {
      const int q = q0 + threadIdx.x, d = min(x.now, (q + 1) * rows) - 1;
      const int stay = __syncthreads_count(q < pieces && src[d] == d);
      first += stay;
      if (stay < kMove) break;
    }
  }
  int next[kRounds];  // keys that this thread copies in the piece that is fetched next
  auto look = [&](int q) {
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      const int d = q * rows + u * step + lead;
      next[u] = busy && d < x.now ? src[d] : -1;
    }
  };
  auto fetch = [&](int q) {
    int page[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) page[u] = next[u] >= 0 ? from[next[u] / kTile] : -1;
    const uint32_t at = place + (q % kStages) * kPieceBytes;
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      if (valid(page[u]))
        copy_async16(at + u * step * words * 16, mine + static_cast<size_t>(page[u]) * page_bytes +
                                                     static_cast<size_t>(next[u] % kTile) * row_bytes);
      else if (next[u] >= 0)  // (an entry that names no page reads zeros)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + u * step * words * 16), "r"(0) : "memory");
    }
    copy_commit();
    look(q + 1);
  };
  look(first);
#pragma unroll 1
  for (int q = first; q < first + kStages - 1; ++q) fetch(q);
#pragma unroll 1
  for (int q = first; q < pieces; ++q) {
    fetch(q + kStages - 1);
    copy_wait<kStages - 1>();
    __syncthreads();  // the piece has been read by all
    const uint32_t at = place + (q % kStages) * kPieceBytes;
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      const int d = q * rows + u * step + lead;
      if (!busy || d >= x.now) continue;
      const int p = to[d / kTile];
      uint4 v;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + u * step * words * 16));
      if (valid(p))
        *reinterpret_cast<uint4*>(mine + static_cast<size_t>(p) * page_bytes + static_cast<size_t>(d % kTile) * row_bytes) = v;
    }
    __syncthreads();  // its place is filled again in the next turn
  }
  copy_wait<0>();
}

// The weights of one (sequence, layer, head): as move_rows, a piece in registers.
__device__ void move_weights(const Cut& x, const int32_t* src, const float* from, float* to, long width) {
  const bool cut = x.now < x.len;
  if (!cut && from == to) return;
  constexpr int U = 8;
  for (int d0 = 0; d0 < x.now; d0 += kMove * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int d = d0 + u * kMove + threadIdx.x;
      v[u] = d < x.now ? from[cut ? src[d] : d] : 0.f;
    }
    __syncthreads();  // all of the piece has been read
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int d = d0 + u * kMove + threadIdx.x;
      if (d < x.now) to[d] = v[u];
    }
  }
  for (long d = x.now + threadIdx.x; d < width; d += kMove) to[d] = 0.f;
}

__global__ void __launch_bounds__(kMove)
    move_kernel(const Call c, const Space w, const Layers layers, const PagePools pools, int per_layer, int slices,
                int state_too) {
  extern __shared__ unsigned char stage[];
  wait_for_previous();
  if (w.head[0] == 0) return;
  const PageState& s = c.s;
  const long width = static_cast<long>(s.max_pages) * kTile;
  const long lists = static_cast<long>(c.n) * c.Hkv;  // of a layer
  const long movers = lists * pools.count * slices;
  long at = blockIdx.x;
  if (at < movers) {
    const int slice = static_cast<int>(at % slices);
    at /= slices;
    const int h = static_cast<int>(at % c.Hkv);
    at /= c.Hkv;
    const int i = static_cast<int>(at % c.n), pool = static_cast<int>(at / c.n);
    const Cut x = w.cut[i];
    if (x.now == x.len || x.now == 0) return;
    const int row_bytes = static_cast<int>(pools.page_bytes / (static_cast<size_t>(c.Hkv) * kTile));
    const int32_t* src = w.src + (pool / per_layer * lists + static_cast<long>(i) * c.Hkv + h) * width;
    const int all = row_bytes / 16, each = (all + slices - 1) / slices;  // 16-byte words of a row, of a slice
    for (int first = slice * each; first < min(all, (slice + 1) * each); first += kMove) {
      move_rows(c, w, pools.base[pool], pools.page_bytes, i, h, src, row_bytes, first * 16,
                min(kMove, min(all, (slice + 1) * each) - first), stage);
      __syncthreads();
    }
    return;
  }
  at -= movers;
  if (at < lists * layers.count) {
    const int h = static_cast<int>(at % c.Hkv), i = static_cast<int>(at / c.Hkv % c.n), layer = static_cast<int>(at / lists);
    const Cut x = w.cut[i];
    const long row = (static_cast<long>(x.row) * c.Hkv + h) * width;
    move_weights(x, w.src + at * width, layers.weights[layer] + row, layers.out[layer] + row, width);
    return;
  }
  at -= lists * layers.count;
  if (!state_too || at >= s.num_rows) return;
  const int row = static_cast<int>(at), i = w.entry[row];
  const int32_t* old = s.table + static_cast<long>(row) * s.max_pages;
  int32_t* now = c.out_table + static_cast<long>(row) * s.max_pages;
  if (i < 0) {  // not listed
    if (now != old)
      for (int j = threadIdx.x; j < s.max_pages; j += kMove) now[j] = old[j];
    if (threadIdx.x == 0 && c.out_lens != s.lens) c.out_lens[row] = s.lens[row];
    return;
  }
  const Cut x = w.cut[i];
  for (int j = threadIdx.x; j < s.max_pages; j += kMove)
    now[j] = j < tiles_of(x.now) ? w.to[static_cast<long>(i) * s.max_pages + j] : -1;
  if (threadIdx.x == 0) c.out_lens[row] = x.now;
}

}  // namespace

size_t evict_workspace(int num_pages, int num_rows, int max_pages, int n, int Hkv, int num_layers, int per_layer) {
  return space_of(nullptr, nullptr, num_pages, num_rows, max_pages, n, Hkv, layers_of_a_launch(num_layers, per_layer));
}

cudaError_t launch_pages_evict(const EvictArgs& a, void* ws, cudaStream_t st) {
  const int group = layers_of_a_launch(a.num_layers, a.per_layer);
  Space w;
  space_of(&w, ws, a.s.num_pages, a.s.num_rows, a.s.max_pages, a.n, a.Hkv, group);
  Call c{a.s, a.rows, a.keep, a.n, a.recent, a.Hkv, a.out_refs, a.out_table, a.out_lens, a.result};
  const int row_words = static_cast<int>(a.page_bytes / (static_cast<size_t>(a.Hkv) * kTile) / 16);
  cudaError_t e = cudaSuccess;
  // (with no sequence listed there is nothing but the state: one pair of launches)
  for (int l0 = a.n > 0 ? 0 : (a.num_layers - 1) / group * group; e == cudaSuccess && l0 < a.num_layers; l0 += group) {
    Layers layers{};
    layers.count = a.num_layers - l0 < group ? a.num_layers - l0 : group;
    PagePools pools{};
    pools.page_bytes = a.page_bytes;
    pools.count = layers.count * a.per_layer;
    for (int l = 0; l < layers.count; ++l) {
      layers.weights[l] = a.weights[l0 + l];
      layers.out[l] = a.out_weights[l0 + l];
    }
    for (int q = 0; q < pools.count; ++q) pools.base[q] = static_cast<unsigned char*>(a.pools[l0 * a.per_layer + q]);
    const bool last = l0 + group >= a.num_layers;
    const long lists = static_cast<long>(a.n) * a.Hkv * layers.count, movers = static_cast<long>(a.n) * a.Hkv * pools.count;
    const int plan_too = l0 == 0 || a.n == 0;
    choose_kernel<<<static_cast<unsigned>(lists + plan_too), kChoose, 0, st>>>(c, w, layers, plan_too);
    if ((e = cudaGetLastError()) != cudaSuccess) break;
    // few movers share their rows' columns, in pieces of 64 bytes at least
    int slices = 1;
    while (movers * slices < 4 * kSMs && row_words % (2 * slices) == 0 && row_words / (2 * slices) >= 4) slices *= 2;
    const long blocks = movers * slices + lists + (last ? a.s.num_rows : 0);
    e = launch_behind(move_kernel, static_cast<unsigned>(blocks), kMove, kStages * kPieceBytes, st, c, w, layers, pools,
                      a.per_layer, slices, static_cast<int>(last));
  }
  return e;
}

}  // namespace ssattn

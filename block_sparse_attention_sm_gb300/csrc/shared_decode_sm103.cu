// Decode over shared pages for sm_103a: one new token a sequence, and pages
// that several sequences hold are read once for all of them; optionally each
// key's attention weight is added to the sequence's record of it.
//
// Mathematics: softmax attention splits over the keys.  With the keys of a
// sequence cut into sets, each gives a reference maximum m, a sum l and an
// unnormalised output O, and o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i with
// M = max m_i.  A node of the plan is such a set for several sequences at once:
// the tiles that they share.  Its rows are the sequences x the G heads of a KV
// head, which makes of the many matrix-vector products of a decode step a
// matrix product: 64 sequences x 4 heads are 256 rows for each key read.
//
// What a sequence has to itself has only G rows.  128 / G sequences are bundled:
// their rows are the 128 rows of the MMAs, their tiles come one behind the other,
// and each tile counts for the rows of its own sequence alone: P.V leaves the other
// lanes of O as they are, whatever the tile's values hold.  So the rows' state stays
// in place while short sequences pass: no new Q and no result to write for each.
//
// Work: an item is (bundle, KV head) or (shared node, KV head, block of up to 256
// rows), as long as it has tiles.  All items' tiles laid end to end are cut into
// equal shares, one a CTA, so that the SMs end together whatever the lengths.
// Every piece of an item writes its rows' (m, l, O) in fp32, and merge_kernel joins
// them.  The cuts follow from the plan and the lengths, which every CTA adds up for
// itself at its start: nothing comes from the host, the lengths may change from step
// to step under the same plan.
//
// One CTA: two streams t = 0, 1, each with scores S_t, weights P_t (bf16, over
// S_t) and output O_t in TMEM (128 columns each of S and O) and a softmax
// warpgroup, one thread a row.  Of more than 128 rows each stream has half, and
// both take every tile.  Of fewer both have the same rows and take alternate tiles:
// the way of a tile from its scores to P.V is longer than the time its bytes take,
// so two are under way at once.  Scores: S_t = Q_t K^T (SS form, K-major, 128-byte swizzle); O_t += P_t V (TS
// form, V MN-major).
//
// Warps 0-3 / 4-7 softmax of stream 0 / 1 (they also load their rows of Q: the
// next piece's before they write this one's result), 8 loads K and V tiles
// through one ring, 9 and 11 issue the MMAs of stream 0 and 1, 10 works out the pieces, in segments
// of up to 16 tiles with a tile's page and sequence each.
//
// The last tile of a sequence, of r < 128 keys, is loaded from row r - 128 of
// its page: zeros come in front, the keys follow, and what the page holds behind
// the sequence's end is never read.
//
// Bound: 64 sequences (32 / 8 heads of 128) on a shared prefix of 32K keys with 100-900 of
// their own take 60 us, 271 MB read: 7 us until the first scores, then the pages at 80% of
// the copy rate (a tile that both streams take: ~3600 cycles, of which scores and P.V issue
// for 1100 a stream and the softmax takes 1450; one of a bundle waits for its bytes).  64
// sequences of 32K each, nothing shared: 1.29 ms, 95%.  Small batches are a chain: ~4 us
// until the first tile is asked for, 2 until its scores, 1.2 a tile.
//
// With weights the raw scores also go to the workspace (4 G bytes a key and KV
// head, beside 4 d of K and V), and when the merge has the row's denominator,
// weigh_kernel adds up exp2(s - lse) over the group's heads.  Each sum is made
// by one thread in the order of the heads: the same from run to run.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "ptx_sm103.cuh"
#include "shared_decode.cuh"

namespace ssattn {

namespace {

constexpr float kSlackLog2 = 40.0f;  // how far weights may be above 1 (exp2 domain)
constexpr int kSMs = 152;
constexpr int kThreads = 384;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpPlan = 10, kWarpMma2 = 11;
constexpr int kRows = 256;      // rows of an item
constexpr int kSegments = 4;    // published segments
constexpr int kSegTiles = 16;
constexpr int kOpeners = 256 + 32;  // softmax warps and planner
// Register split (see the prefill kernel): the launch's pool, exactly.
constexpr int kLaunchRegs = 168, kRegsIssue = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax == kThreads * kLaunchRegs, "register split");

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kRing = (D == 128) ? 5 : 10;
  static constexpr int kRingOff = 2 * kTileBytes;  // behind the two Q tiles
  static constexpr int kCtlOff = kRingOff + kRing * kTileBytes;
  static constexpr int kCtlBytes = 2048;
  static constexpr int kSmemBytes = kCtlOff + kCtlBytes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
  // The sums over the batch are made where the tiles come later: a place's tiles
  // (4 bytes), a shared node's cost and rows (12 bytes).
  static_assert(4 * (kSharedMaxB + 2) <= kCtlOff && 8 * (kPlanMaxB + 1) + 8 * kPlanMaxB <= kCtlOff, "sums");
};

// Eight floats at once (32 bytes, a whole sector of a line), 32-byte aligned.
__device__ __forceinline__ void store8(float* to, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The tiles [t0, t1) of places [first, first + count).
struct Node {
  int first, count, t0, t1;
};

// A tile: where it lies in the pools, which of its sequence's it is, the zero rows in
// front of its keys, whose rows it counts for (a place of the bundle; -1: all).
struct Tile {
  int z, tile;
  short shift, place;
};

// Up to kSegTiles consecutive tiles of a piece (a run of tiles of one item).
struct Segment {
  short n;            // tiles; 0: no more segments
  short odd;          // tiles of the piece in front of the segment's, modulo 2
  short start, end;   // the piece's first / last segment
  int kvh;
  int first;          // the item's first place
  int row0;           // its first row among the node's (place x head of the group)
  short rows;         // its rows
  short both;         // each stream has half the rows and takes every tile; else all rows, alternate tiles
  long long out;      // its first partial row (-1: no room)
  Tile tile[kSegTiles];
};

struct Ctl {
  uint64_t r_full[10], r_empty[10];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t turn[2], mma_done[2];
  uint32_t tmem_base;
  int abort_flag;
  int n_issued;
  uint32_t leaf_total, total;  // cost of all bundles, of all items
  uint32_t least;                // a share's least cost
  Segment seg[kSegments];
};

__device__ __forceinline__ const int32_t* valid_plan(const SharedParams& p) {
  const int32_t* plan = p.plan;
  if (plan != nullptr && (plan[0] != p.B || plan[1] != p.max_pages || plan[2] != kPlanMark)) plan = nullptr;
  return plan;
}
__device__ __forceinline__ int place_of(const int32_t* plan, int i, int B) {
  return plan != nullptr ? max(0, min(B - 1, plan[kPlanHead + i])) : i;
}
__device__ __forceinline__ int length_of(const SharedParams& p, int b) {
  return max(0, min(p.lens[b], p.max_pages * kTile));
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Node n of 2 B (without a plan: B).
__device__ __forceinline__ Node node_of(const SharedParams& p, const int32_t* plan, int n) {
  Node x{n, 1, 0, 0};
  if (plan == nullptr) {
    x.t1 = tiles_of(length_of(p, n));
    return x;
  }
  const int32_t* w = plan + kPlanHead + p.B + static_cast<long>(n) * kNodeWords;
  if (n < p.B) {
    x.t1 = tiles_of(length_of(p, place_of(plan, n, p.B)));
    x.t0 = max(0, min(w[2], x.t1));
  } else {
    x.first = max(0, min(w[0], p.B - 1));
    x.count = max(0, min(w[1], p.B - x.first));
    x.t0 = max(0, min(w[2], p.max_pages));
    x.t1 = max(x.t0, min(w[3], p.max_pages));
    if (x.count == 0) x.t1 = x.t0;
  }
  return x;
}

// How a node's rows are dealt to items (whole places), and an item's rows in the partial results.
struct Deal {
  int blocks, rows;   // items a KV head, rows of an item (the last may have fewer)
  int part;           // partial rows of a piece: two results each where the streams take alternate tiles
};
__device__ __forceinline__ Deal deal_of(const Node& x, int G) {
  Deal d{1, x.count * G, 0};
  if (d.rows > kRows) {
    const int most = kRows / G;
    d.blocks = (x.count + most - 1) / most;
    d.rows = (x.count + d.blocks - 1) / d.blocks * G;
  }
  d.part = d.rows <= kTile ? 2 * d.rows : d.rows;
  return d;
}

// Costs, in the shares of the CTAs: 1 for a tile of a bundle; where both streams take
// every tile it is about twice that (2:3, 4:7, 1:2, 5:11 and 1:1 give 337, 331, 317, 320 and 379 us at
// four layers of 64 sequences on a prefix of 32K keys).  An item costs kItemCost in front of
// its first tile: a CTA that goes on to another one ends ~2 us later than the others
// (0, 1, 2, 3, 4, 8: 299, 287, 291, 279, 279, 284 us there, and 3 of 24 us with 8 sequences of 2K).
constexpr int kItemCost = 3;
// (With weights each of the rows writes its scores: three times; 64 sequences on 8K keys 2, 3, 4: 95, 88, 86 us,
// 24 on 8K 43, 41, 46.)
__device__ __forceinline__ int both_cost(const SharedParams& p) { return p.scores != nullptr ? 3 : 2; }
__device__ __forceinline__ int cost_of(const SharedParams& p, const Deal& d) { return d.rows > kTile ? both_cost(p) : 1; }
// A CTA's share of all items' cost: at least a tile of any kind (`least`), so that each CTA
// between an item's first and last has a part of it.  Costs fit 32 bits (kMaxSharedTiles).
__device__ __forceinline__ uint32_t share_of(uint32_t total, uint32_t ctas, uint32_t least) {
  return max(least, (total + ctas - 1) / ctas);
}

// What the places below a place have: own tiles, cost and partial rows of their shared nodes.
struct Sums {
  uint32_t tiles, cost;
  long long rows;
  __device__ __forceinline__ void add(const Sums& x) { tiles += x.tiles, cost += x.cost, rows += x.rows; }
};
// Exclusive sums over the block's first `used` threads, in place; returns the total.
__device__ Sums block_sums(Sums& v, int used, bool nodes, Sums* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (used + 31) / 32;
  const Sums mine = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sums x{__shfl_up_sync(0xffffffffu, v.tiles, o), 0, 0};
    if (nodes) {
      x.cost = __shfl_up_sync(0xffffffffu, v.cost, o);
      x.rows = __shfl_up_sync(0xffffffffu, v.rows, o);
    }
    if (lane >= o) v.add(x);
  }
  if (lane == 31 && warp < warps) scratch[warp] = v;
  __syncthreads();
  v.tiles -= mine.tiles, v.cost -= mine.cost, v.rows -= mine.rows;
  Sums all{0, 0, 0};
#pragma unroll 1
  for (int w = 0; w < warps; ++w) {
    const Sums x = scratch[w];
    if (w < warp) v.add(x);
    all.add(x);
  }
  __syncthreads();
  return all;
}

// (A launch's code comes out of L2 line by line: waits, divisions and the parts of a
// piece appear once each, and loops that need not be unrolled are not.)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    shared_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const SharedParams p) {
  using C = Cfg<D>;
  constexpr int NR = C::kRing;
  static_assert(sizeof(Ctl) <= C::kCtlBytes, "control block overflow");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sR = smem + C::kRingOff;
  auto* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  volatile int* abort_flag = &ctl->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.B, G = p.G, nb = kTile / G;  // sequences of a bundle
  let_next_start();

  if (tid < NR) {
    mbar_init(&ctl->r_full[tid], 1);
    mbar_init(&ctl->r_empty[tid], 2);  // both issuers
  } else if (tid >= 32 && tid < 32 + kSegments) {
    mbar_init(&ctl->seg_full[tid - 32], 1);
    mbar_init(&ctl->seg_empty[tid - 32], 11);  // softmax warps, loader, issuers
  } else if (tid >= 64 && tid < 66) {
    const int t = tid - 64;
    mbar_init(&ctl->q_full[t], 4);
    mbar_init(&ctl->s_full[t], 1);
    mbar_init(&ctl->p_full[t], 4);
    mbar_init(&ctl->o_full[t], 1);
    mbar_init(&ctl->o_free[t], 4);
    mbar_init(&ctl->turn[t], 1);
    mbar_init(&ctl->mma_done[t], 1);
    if (t == 0) {
      ctl->abort_flag = 0;
      ctl->n_issued = 0;
    }
  }
  fence_mbar_init();
  if (warp == kWarpMma) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  wait_for_previous();
  const int32_t* plan = valid_plan(p);
  const int nodes = plan != nullptr ? B : 0;  // shared ones
  // Sums over the batch, in the shared memory that the tiles take later: the own
  // tiles of the places below each, the cost and partial rows of the shared nodes
  // below each.
  uint32_t* cum = reinterpret_cast<uint32_t*>(smem);                                     // [B + 1]
  uint32_t* node_at = cum + B + 1;                                                       // [nodes]
  long long* node_rows = reinterpret_cast<long long*>(smem + (4 * (2 * B + 1) + 7) / 8 * 8);  // [nodes]
  {
    const int each = (B + kThreads - 1) / kThreads, n0 = min(B, tid * each), n1 = min(B, n0 + each);
    Sums v{0, 0, 0}, all{0, 0, 0};
    Node x{}, y{};
    Deal d{};
    bool wide = false;  // a node of more than 128 rows
    auto leaf_cost = [&](uint32_t tiles) { return (tiles + kItemCost * ((B + nb - 1) / nb)) * p.Hkv; };
    // twice: adding up, then (with what lies below) writing
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
      for (int n = n0; n < n1; ++n) {
        if (pass == 0 || each > 1) {
          x = node_of(p, plan, n);
          if (plan != nullptr) {
            y = node_of(p, plan, B + n);
            d = deal_of(y, G);
          }
        }
        if (pass == 1) {
          cum[n] = v.tiles;
          if (plan != nullptr) {
            node_at[n] = leaf_cost(all.tiles) + v.cost;
            node_rows[n] = 2ll * p.Hq * B + v.rows;
          }
        }
        v.tiles += x.t1 - x.t0;
        if (y.t1 > y.t0) {
          wide |= d.rows > kTile;
          v.cost += ((y.t1 - y.t0) * cost_of(p, d) + kItemCost) * d.blocks * p.Hkv;
          v.rows += static_cast<long long>(d.blocks) * p.Hkv * d.part;
        }
      }
      if (pass == 0) all = block_sums(v, (B + each - 1) / each, plan != nullptr, reinterpret_cast<Sums*>(ctl->seg));
    }
    wide = __syncthreads_or(wide);
    if (tid == 0) {
      ctl->least = wide ? both_cost(p) : 2;  // (two tiles of a bundle: a stream each)
      cum[B] = all.tiles;
      ctl->leaf_total = leaf_cost(all.tiles);
      ctl->total = ctl->leaf_total + all.cost;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_small(bar, parity, abort_flag); };
  // Segment number k, when it has been published (its place is given back by `seg_done`).
  auto seg_at = [&](int k) -> const Segment* {
    return wait(&ctl->seg_full[k % kSegments], (k / kSegments) & 1) ? &ctl->seg[k % kSegments] : nullptr;
  };
  auto seg_done = [&](int k) { mbar_arrive(&ctl->seg_empty[k % kSegments]); };

  if (warp >= 8) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == kWarpLoad) {
      // ---------------------------------------------------------- loader
      // Order of use: K0 V0 K1 V1 .. where both streams take every tile,
      // K0 K1 V0 K2 V1 .. where they alternate.
      if (lane == 0) {
        uint32_t slot = 0, par = 1;
        int e = 0;
        Tile held{};  // the tile whose V comes next
        bool ok = true;
#pragma unroll 1
        for (int k = 0; ok; ++k) {
          const Segment* x = seg_at(k);
          if (x == nullptr || x->n == 0) break;
          const int n = x->n, both = x->both, steps = n + (!both && x->end), first = !both && x->start;
#pragma unroll 1
          for (int i = 0; ok && i < steps; ++i) {
            const Tile d = i < n ? x->tile[i] : held;
#pragma unroll 1
            for (int v = 0; ok && v < 2; ++v) {
              if (v == 0 ? i >= n : first && i == 0) continue;
              const Tile y = v == 0 || both ? d : held;
              if (!(ok = wait(&ctl->r_empty[slot], par))) break;
              mbar_arrive_expect_tx(&ctl->r_full[slot], C::kTileBytes);
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(sR + slot * C::kTileBytes + c * 16384, v == 0 ? &tmK : &tmV, &ctl->r_full[slot], c * 64,
                            -y.shift, y.z);
              *reinterpret_cast<volatile int*>(&ctl->n_issued) = ++e;
              if (++slot == NR) slot = 0, par ^= 1;
            }
            held = d;
          }
          seg_done(k);
        }
      }
      __syncwarp();
    } else if (warp == kWarpMma || warp == kWarpMma2) {
      // ---------------------------------------------------------- MMAs of stream t
      // A stream's turn: P.V of its last tile and the scores of its next.  The issuers
      // take turns (`turn`), so that one softmax runs beside the other stream's MMAs
      // (left alone both fell into step: 4700 cycles a tile), and there are two so that
      // one's waits and commits run beside the other's MMAs (a single issuer: 4400).
      // Both pass every entry of the ring in order, those of the other stream too.
      {  // (a whole warp, one lane of which issues: what the MMAs are given stays uniform)
        const int t = __shfl_sync(0xffffffffu, warp == kWarpMma ? 0 : 1, 0);
        auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);
        const uint64_t dq = smem_desc(smem_u32(sQ) + t * C::kTileBytes, 16, 1024);
        const uint64_t dk0 = smem_desc(smem_u32(sR), 16, 1024), dv0 = smem_desc(smem_u32(sR), 16384, 1024);
        const uint32_t colS = tmem + C::kColS + 128 * t, colO = tmem + C::kColO + 128 * t;
        uint32_t slot = 0, par = 0;
        uint32_t qn = 0, pn = 0, on = 1, tn = t ^ 1;  // parities
        auto next = [&]() {
          if (++slot == NR) slot = 0, par ^= 1;
        };
        bool ok = true;
        // A bundle: the places of the stream's last tile and of the one whose P.V was last.
        int place = -1, before = -1;
        uint32_t off[4] = {0, 0, 0, 0};  // lanes that the stream's last tile does not count for
#pragma unroll 1
        for (int k = 0, u = 0; ok; ++k) {
          if (!wwait(&ctl->seg_full[k % kSegments], (k / kSegments) & 1)) break;
          const Segment* x = &ctl->seg[k % kSegments];
          if (x->n == 0) break;
          // P.V follows its scores by one tile (both streams) or two (alternate ones).
          const int n = x->n, both = x->both, lag = both ? 1 : 2, last = x->end;
          if (x->start != 0) u = 0;
          const int u0 = u, end = u + n;            // tiles up to the segment's end
          const int steps = last ? (both ? end + 1 : (end + 3) & ~1) : end;
          const bool bundle = x->tile[0].place >= 0;
#pragma unroll 1
          for (; ok && u < steps; ++u) {
            const bool mine = both || (u & 1) == t, has_v = u >= lag && u < end + lag, has_k = u < end;
            if (!mine) {
#pragma unroll 1
              for (int e = has_v + has_k; ok && e > 0; --e) {
                ok = wwait(&ctl->r_full[slot], par);
                if (elect_one()) mbar_arrive(&ctl->r_empty[slot]);
                __syncwarp();
                next();
              }
              continue;
            }
            // The tiles are waited for in front of the turn, the weights last: they come latest.
            const bool first = u < 2 * lag, begins = first || place != before;
            const uint32_t slot_v = slot, slot_k = !has_v ? slot : slot + 1 == NR ? 0 : slot + 1;
            if (has_v) {
              if (!(ok = wwait(&ctl->r_full[slot], par))) break;
              next();
              before = place;
            }
            if (has_k) {
              if (!(ok = wwait(&ctl->r_full[slot], par))) break;
              next();
              if (u < lag) {
                if (!(ok = wwait(&ctl->q_full[t], qn))) break;
                qn ^= 1;
              }
            }
            if (!(ok = wwait(&ctl->turn[t], tn))) break;
            tn ^= 1;
            if (has_v) {
              if (first) {  // the piece before has been read out of O
                if (!(ok = wwait(&ctl->o_free[t], on))) break;
                on ^= 1;
              }
              if (!(ok = wwait(&ctl->p_full[t], pn))) break;
              pn ^= 1;
            }
            tc_fence_after();
            if (has_v) {  // O_t += P_t V
              const uint64_t dv = dv0 + slot_v * (C::kTileBytes >> 4);
              if (elect_one()) {
                if (bundle) {
#pragma unroll
                  for (int kk = 0; kk < kTile / 16; ++kk)
                    mma_bf16_ts_lanes(colO, colS + kk * 8, dv + ((kk * 2048) >> 4), idO, off, (!begins || kk > 0) ? 1u : 0u);
                } else {
#pragma unroll
                  for (int kk = 0; kk < kTile / 16; ++kk)
                    mma_bf16_ts(colO, colS + kk * 8, dv + ((kk * 2048) >> 4), idO, (!first || kk > 0) ? 1u : 0u);
                }
                if (u >= end) mma_commit(&ctl->o_full[t]);
                mma_commit(&ctl->r_empty[slot_v]);
              }
              __syncwarp();
            }
            if (has_k) {  // S_t = Q_t K^T
              // (S_t was read before P_t was handed over: the fence in front of P.V covers it)
              const uint64_t dk = dk0 + slot_k * (C::kTileBytes >> 4);
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                  mma_bf16_ss(colS, dq + off, dk + off, idS, kk > 0 ? 1u : 0u);
                }
                mma_commit(&ctl->s_full[t]);
              }
              __syncwarp();
            }
            if (elect_one()) {
              mbar_arrive(&ctl->turn[t ^ 1]);
              if (has_k) mma_commit(&ctl->r_empty[slot_k]);
            }
            __syncwarp();
            if (has_k && bundle) {
              // (Behind the turn, where it costs no time.)  A bundle's tile counts for the
              // rows of one sequence: P.V leaves the others' lanes as they are, whatever
              // the tile's values hold, and the sequence's first tile begins its O.
              place = x->tile[u - u0].place;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int lo = max(0, place * G - 32 * w), hi = min(32, place * G + G - 32 * w);
                off[w] = hi > lo ? ~((0xffffffffu >> (32 - (hi - lo))) << lo) : 0xffffffffu;
              }
            }
          }
          __syncwarp();
          if (elect_one()) seg_done(k);
          __syncwarp();
        }
        if (elect_one()) {
          mma_commit(&ctl->mma_done[t]);
          mbar_wait(&ctl->mma_done[t], 0, nullptr);
        }
      }
      __syncwarp();
    } else if (warp == kWarpPlan) {
      // ---------------------------------------------------------- pieces
      // A tile belongs to the CTA whose share its cost begins in.
      const uint32_t leaf_total = ctl->leaf_total, total = ctl->total, per = share_of(total, gridDim.x, ctl->least);
      uint32_t at = min(total, per * blockIdx.x);
      const uint32_t end = min(at + per, total);
      // Where the share begins: in a bundle ..
      int j = 0, kvh = 0, base = 0, T = 0, skip = 0;  // bundle, head, its first place's sum, its tiles, those in front
      int n = 0;                                      // .. or a shared node
      uint32_t n_at = 0;
      long long n_rows = 0;
      auto tile_at = [&] {  // cost in front of tile `skip` of the item
        return static_cast<uint32_t>(base + kItemCost * j) * p.Hkv + static_cast<uint32_t>(kvh) * (T + kItemCost) + kItemCost + skip;
      };
      if (at < end) {
        const bool leaf = at < leaf_total;
        int lo = 0, hi = leaf ? (B + nb - 1) / nb : nodes;
#pragma unroll 1
        while (hi - lo > 1) {  // the last one that begins at or below `at` (an empty one: the next begins there too)
          const int mid = (lo + hi) / 2;
          if ((leaf ? (cum[mid * nb] + kItemCost * mid) * p.Hkv : node_at[mid]) <= at) lo = mid; else hi = mid;
        }
        if (leaf) {
          j = lo;
          base = cum[j * nb];
          T = cum[min(B, (j + 1) * nb)] - base;
          const uint32_t in = at - static_cast<uint32_t>(base + kItemCost * j) * p.Hkv;
          kvh = in / (T + kItemCost);
          skip = max(0, static_cast<int>(in - static_cast<uint32_t>(kvh) * (T + kItemCost)) - kItemCost);
          at = tile_at();
        } else {
          n = lo;
        }
        n_at = nodes > 0 ? node_at[n] : 0;
        n_rows = nodes > 0 ? node_rows[n] : 0;
      }
      // The piece that is being published, and of a bundle 32 places, a lane each.
      Segment seg{};
      int left = 0, done = 0;             // its tiles to come, its tiles published
      int t_first = 0, node_b = 0;        // a node's piece: its first tile, a sequence that has them
      bool bundle = false;
      int w0 = 0, before = 0, window = 0; // window: first place, tiles in front of it, its tiles
      int b = 0, t0 = 0, count = 0, len = 0, sum = 0;
      bool ok = true, opened = false;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        // ---- the next piece
#pragma unroll 1
        while (left == 0 && at < end) {
          done = 0;
          if (at < leaf_total) {
            if (skip >= T) {  // the next head's, or the next bundle that has tiles
              if (T == 0 || ++kvh == p.Hkv) {
                kvh = 0;
                base += T;
                if (++j * nb >= B) {  // (no more)
                  at = leaf_total;
                  continue;
                }
                T = 0;
#pragma unroll 1
                for (int i = j * nb + lane; i < min(B, (j + 1) * nb); i += 32) {
                  const Node x = node_of(p, plan, i);
                  T += x.t1 - x.t0;
                }
                T = __reduce_add_sync(0xffffffffu, T);
              }
              skip = 0;
              at = tile_at();
              continue;
            }
            const int first = j * nb, places = min(nb, B - first), rows = places * G;
            bundle = true;
            seg.kvh = kvh;
            seg.first = first;
            seg.row0 = 0;
            seg.rows = static_cast<short>(rows);
            seg.both = 0;
            seg.out = 2ll * G * p.Hkv * first + 2ll * kvh * rows + static_cast<long long>(blockIdx.x) * kRows;
            if (seg.out + 2 * rows > p.part_rows) seg.out = -1;
            left = min(T - skip, static_cast<int>(end - at));
            at += left;
            w0 = -32, before = window = 0;
          } else {
            const Node x = node_of(p, plan, B + n);
            const Deal d = deal_of(x, G);
            const uint32_t Tn = x.t1 - x.t0, cost = cost_of(p, d), each = Tn * cost + kItemCost;
            const uint32_t items = Tn > 0 ? d.blocks * p.Hkv : 0, in = at > n_at ? at - n_at : 0;
            uint32_t item = in / each, u = 0;
            if (in > item * each + kItemCost) u = (in - item * each - kItemCost + cost - 1) / cost;
            if (u >= Tn) u = 0, ++item;  // (the share begins in the item's last tile)
            if (item >= items) {
              n_at += items * each;
              at = max(at, n_at);
              n_rows += static_cast<long long>(items) * d.part;
              if (++n >= nodes) at = end;
              continue;
            }
            at = n_at + item * each + kItemCost + u * cost;
            if (at >= end) break;
            const int head = item / d.blocks;
            bundle = false;
            seg.kvh = head;
            seg.first = x.first;
            seg.row0 = (item - head * d.blocks) * d.rows;
            seg.rows = static_cast<short>(min(d.rows, x.count * G - seg.row0));
            seg.both = d.rows > kTile;
            seg.out = n_rows + static_cast<long long>(item) * d.part + static_cast<long long>(blockIdx.x) * kRows;
            if (seg.out + d.part > p.part_rows) seg.out = -1;
            t_first = x.t0 + u;
            node_b = place_of(plan, x.first, B);
            left = min(Tn - u, (end - at + cost - 1) / cost);
            at += left * cost;
          }
        }
        // ---- its next tiles, a lane each
        int m = min(kSegTiles, left);
        Tile d{0, 0, 0, -1};
        if (m > 0) {
          int seq = node_b;
          d.tile = t_first + done + lane;
          if (bundle) {
            const int places = min(nb, B - seg.first);
#pragma unroll 1
            while (skip + done >= before + window && w0 + 32 < places) {  // on to the window of 32 places that has them
              before += window;
              w0 += 32;
              b = t0 = count = len = 0;
              if (w0 + lane < places) {
                const Node x = node_of(p, plan, seg.first + w0 + lane);
                b = place_of(plan, seg.first + w0 + lane, B);
                len = length_of(p, b);
                t0 = x.t0;
                count = x.t1 - x.t0;
              }
              sum = count;
#pragma unroll 1
              for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
              }
              window = __shfl_sync(0xffffffffu, sum, 31);
            }
            const int want = skip + done - before;  // of the window's
            m = max(0, min(m, window - want));
            if (m == 0) left = 0;  // (lengths that changed under the call)
            // the place of tile want + lane: the first whose sum is above it
            const int x = min(want + lane, window - 1);
            int q = 0;
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1)
              if (__shfl_sync(0xffffffffu, sum, q + o - 1) <= x) q += o;
            seq = __shfl_sync(0xffffffffu, b, q);
            d.tile = __shfl_sync(0xffffffffu, t0, q) + x -
                     (__shfl_sync(0xffffffffu, sum, q) - __shfl_sync(0xffffffffu, count, q));
            d.shift = static_cast<short>(max(0, (d.tile + 1) * kTile - __shfl_sync(0xffffffffu, len, q)));
            d.place = static_cast<short>(w0 + q);
          }
          if (lane < m) {
            const int page = p.table[static_cast<long>(seq) * p.max_pages + d.tile];
            d.z = page >= 0 && page < p.num_pages ? page * p.Hkv + seg.kvh : p.num_pages * p.Hkv;
          }
          if (m == 0) {
            --k;
            continue;
          }
        }
        // ---- published (without tiles: the end)
        if (!opened) barrier_sync(2, kOpeners);  // from here on the tiles may land over the sums
        opened = true;
        ok = __all_sync(0xffffffffu, wait(&ctl->seg_empty[k % kSegments], ((k / kSegments) & 1) ^ 1));
        if (!ok) break;
        Segment& to = ctl->seg[k % kSegments];
        if (lane < m) to.tile[lane] = d;
        if (lane == 0) {
          to.n = static_cast<short>(m);
          to.odd = static_cast<short>(done & 1);
          to.start = done == 0;
          to.end = m == left;
          to.kvh = seg.kvh;
          to.first = seg.first;
          to.row0 = seg.row0;
          to.rows = seg.rows;
          to.both = seg.both;
          to.out = seg.out;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->seg_full[k % kSegments]);
        if (m == 0) break;
        done += m;
        left -= m;
        if (left == 0 && bundle) skip += done;
      }
    }
    if (warp == kWarpLoad && lane == 0 && *abort_flag) {
      // let the copies in flight land before shared memory is released
      const int n = *reinterpret_cast<volatile int*>(&ctl->n_issued);
#pragma unroll 1
      for (int s = 0; s < NR; ++s)
        if (n > s) mbar_wait(&ctl->r_full[s], ((n - 1 - s) / NR) & 1, nullptr);
    }
    __syncwarp();
    tc_fence_before();
    barrier_sync(1, kThreads);
    if (warp == kWarpMma) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, C::kTmemCols);
    }
  } else {
    // ---------------------------------------------------------- softmax of stream t
    setmaxnreg_inc<kRegsSoftmax>();
    const int t = warp >> 2, row = tid & 127, w0 = (warp & 3) * 32;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(w0) << 16);
    const uint32_t colS = lane_base + C::kColS + 128 * t, colO = lane_base + C::kColO + 128 * t;
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f32x2(sl2, sl2);
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
    auto place_row = [&](int r) { return p.inv_g != 0 ? static_cast<int>(__umulhi(r, p.inv_g)) : r; };  // r / G
    {  // Where the merge finds the results of a (place, KV head): this CTA's part of the list, while there is nothing else to do.
      const int levels = plan != nullptr ? 1 + kPlanLevels : 1, all = B * p.Hkv * levels;
      const uint32_t per = share_of(ctl->total, gridDim.x, ctl->least);
#pragma unroll 1
      for (int e = blockIdx.x * 256 + tid; e < all; e += gridDim.x * 256) {
        const int level = e & (levels - 1), r = plan != nullptr ? e / (1 + kPlanLevels) : e, i = r / p.Hkv, kvh = r - i * p.Hkv;
        Parts x{0, 0, 0};
        uint32_t a = 0, z = 0;  // cost in front of the row's first tile, of its last
        if (level == 0) {
          const int j = i / nb, j0 = j * nb, places = min(nb, B - j0);
          const uint32_t base = cum[j0], T = cum[j0 + places] - base, c0 = cum[i], n = cum[i + 1] - c0;
          if (n > 0) {
            a = (base + kItemCost * j) * p.Hkv + kvh * (T + kItemCost) + kItemCost + (c0 - base);
            z = a + n - 1;
            x.row = 2ll * G * p.Hkv * j0 + (2ll * kvh * places + (i - j0)) * G;
            x.second = places * G;
            x.count = 1;
          }
        } else {
          const int n = plan[kPlanHead + B + 2l * B * kNodeWords + static_cast<long>(i) * kPlanLevels + level - 1];
          if (n >= B && n < 2 * B) {
            const Node y = node_of(p, plan, n);
            const int T = y.t1 - y.t0, place = i - y.first;
            if (T > 0 && place >= 0 && place < y.count) {
              const Deal d = deal_of(y, G);
              const int blk = d.blocks > 1 ? place * G / d.rows : 0, item = kvh * d.blocks + blk, cost = cost_of(p, d);
              a = node_at[n - B] + item * (T * cost + kItemCost) + kItemCost;
              z = a + (T - 1) * cost;
              x.row = node_rows[n - B] + static_cast<long long>(item) * d.part + (place * G - blk * d.rows);
              x.second = d.rows > kTile ? 0 : d.rows;
              x.count = 1;
            }
          }
        }
        if (x.count > 0) {
          const int c0 = a / per, c1 = z / per;
          x.row += static_cast<long long>(c0) * kRows;
          x.count = max(0, min(p.ctas, c1 - c0 + 1)) * (x.second > 0 ? 2 : 1);
        }
        p.parts[e] = x;
      }
      barrier_sync(2, kOpeners);
    }
    uint32_t ns = 0, no = 0;
    int k = 0;
    bool ok = wwait(&ctl->seg_full[0], 0);
    // What the piece before left to be written.
    bool any = false, mine = false, warp_live = false;
    float m_used = -INFINITY, l = 0.f;
    long long out = -1;
#pragma unroll 1
    for (bool open = false; ok; open = true) {
      const Segment* x = &ctl->seg[k % kSegments];
      const int n_first = x->n, both = x->both, rows = x->rows, kvh = x->kvh, place0 = x->first, row0 = x->row0;
      const int half = (rows + 1) / 2, skip = both && t == 1 ? half : 0;  // this stream's first row among the item's
      const int n_rows = !both ? rows : t == 0 ? half : rows - half;
      // The stream's score MMAs of the piece before are done, its Q tile is free: 16-byte
      // word j of row i goes to word j ^ (i & 7) of its 128-byte rows.
      if (n_first > 0 && (t == 0 || both || n_first > 1 || !x->end)) {
        constexpr int W = D / 8, RS = 128 / W;  // words of a row, rows a pass
        const int j = row % W;
        uint8_t* to = sQ + t * C::kTileBytes + (j >> 3) * 16384;
#pragma unroll 1
        for (int i0 = row / W; i0 < n_rows; i0 += 8 * RS) {  // (8 rows in flight)
          uint4 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int r = row0 + skip + min(i0 + u * RS, n_rows - 1), place = place_row(r);
            v[u] = *reinterpret_cast<const uint4*>(p.q + place_of(plan, place0 + place, B) * p.q_stride +
                                                   static_cast<long>(kvh * G + (r - place * G)) * D + j * 8);
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * RS;
            if (i < n_rows) *reinterpret_cast<uint4*>(to + i * 128 + (((j & 7) ^ (i & 7)) << 4)) = v[u];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->q_full[t]);
      }
      if (open) {  // the piece before: its rows' results
        if (any) {
          if (!(ok = wwait(&ctl->o_full[t], no & 1))) break;
          ++no;
        }
        if (warp_live && out >= 0) {
          const bool some = mine && !(m_used == -INFINITY && l == 0.f);  // (a row of NaN has a sum of NaN)
          if (any) {
            tc_fence_after();
            const uint32_t all = __ballot_sync(0xffffffffu, some);
            if (__popc(all) <= 8) {  // few rows: as they lie, 32 bytes a lane at a time
              float* to = p.part_o + out * D;
#pragma unroll 1
              for (int c = 0; c < D && all != 0; c += 32) {
                uint32_t o[32];
                tmem_ld32p(colO + c, o);
                tmem_wait_ld();
                if (some)
#pragma unroll
                  for (int e = 0; e < 32; e += 8) store8(to + c + e, o + e);
              }
            } else {
              // 32 columns at a time: eight lanes turn their rows' eight 16-byte words around
              // (word j of row i to lane j), so that they write whole 128-byte lines.
              const long long first = out - (lane & 7);
              const uint32_t live = all >> (lane & 24);  // of the eight lanes' rows
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32p(colO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int h = 1; h < 8; h <<= 1) {
                  const bool upper = (lane & h) != 0;
#pragma unroll
                  for (int w = 0; w < 8; ++w) {
                    if (w & h) continue;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      uint32_t &lo = o[4 * w + e], &hi = o[4 * (w | h) + e];
                      const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? lo : hi, h);
                      if (upper) lo = got; else hi = got;
                    }
                  }
                }
                float* to = p.part_o + first * D + c + 4 * (lane & 7);
#pragma unroll
                for (int w = 0; w < 8; ++w)
                  if ((live >> w) & 1u)
                    *reinterpret_cast<uint4*>(to + w * D) = make_uint4(o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]);
              }
            }
          }
          if (mine) p.part_ml[out] = make_float2(m_used == -INFINITY ? -INFINITY : m_used * sl2, l);
        }
        if (any) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->o_free[t]);
        }
      }
      if (n_first == 0) break;
      mine = row < n_rows;
      warp_live = w0 < n_rows;
      out = x->out;
      if (out >= 0) out += skip + row + (!both && t == 1 ? rows : 0);
      const int my_row = row0 + skip + row, my_place = place_row(my_row);
      float* dump = nullptr;  // this row's scores in the workspace
      if (p.scores != nullptr && mine)
        dump = p.scores + (static_cast<size_t>(place_of(plan, place0 + my_place, B)) * p.Hq + kvh * G +
                           (my_row - my_place * G)) * p.max_pages * kTile;
      m_used = -INFINITY;
      l = 0.f;
      any = false;  // the stream has had a tile
#pragma unroll 1
      for (bool last = false; !last;) {
        x = &ctl->seg[k % kSegments];
        const int n = x->n;
        last = x->end != 0;
#pragma unroll 1
        for (int i = both ? 0 : (t + x->odd) & 1; i < n; i += both ? 1 : 2) {
          if (!(ok = wwait(&ctl->s_full[t], ns & 1))) break;
          ++ns;
          const Tile d = x->tile[i];
          // A bundle's tile counts for the rows of one sequence.
          const bool counts = mine && (d.place < 0 || d.place == my_place);
          if (__any_sync(0xffffffffu, counts)) {
            uint32_t sr[128];
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32p(colS + 32 * c, sr + 32 * c);
            tmem_wait_ld();
            if (dump != nullptr && counts) {
              float* to = dump + static_cast<size_t>(d.tile) * kTile;
#pragma unroll
              for (int c = 0; c < 16; ++c) store8(to + 8 * c, sr + 8 * c);
            }
            if (d.shift > 0) {  // columns without a key
#pragma unroll
              for (int e = 0; e < 128; ++e)
                if (e < d.shift) sr[e] = __float_as_uint(-INFINITY);
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 64; ++e)
              mx[e & 3] = fmax3(mx[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // m, the row's reference, is the maximum of its first tile as long as no
            // score is above it by more than 2^kSlackLog2 (bf16 and fp32 have the
            // range, and no precision is lost).
            float alpha = 1.f;
            if (counts) {
              if (m_used == -INFINITY) {
                m_used = top;
              } else if ((top - m_used) * sl2 > kSlackLog2) {
                alpha = ex2_approx((m_used - top) * sl2);
                m_used = top;
                l *= alpha;
              }
            }
            if (__any_sync(0xffffffffu, alpha != 1.f) && any) {
              // (the scores' commit covers P.V of the stream's step before)
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t orr[16];
                tmem_ld16p(colO + c, orr);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                tmem_st16(colO + c, orr);
              }
            }
            // P = exp2(s * scale * log2e - m), rounded to bf16 for P.V (2^-8 of a
            // weight); l adds up the unrounded ones.  (The maximum formed beside the
            // exponentials, with a second turn where it was too low, was slower.)
            const float mb = (m_used == -INFINITY) ? 0.f : m_used * sl2;
            const uint64_t nmb = f32x2(-mb, -mb);
            uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              const uint64_t xp =
                  fma_f32x2(f32x2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), sl2x2, nmb);
              const float p0 = ex2_approx(f32x2_lo(xp)), p1 = ex2_approx(f32x2_hi(xp));
              ls[c & 1] = add_f32x2(ls[c & 1], f32x2(p0, p1));
              sr[c] = pack_bf16x2(p0, p1);
            }
            const uint64_t lsum = add_f32x2(ls[0], ls[1]);
            if (counts) l += f32x2_lo(lsum) + f32x2_hi(lsum);
            tmem_st32p(colS, sr);
            tmem_st32p(colS + 32, sr + 32);
            tmem_wait_st();
            tc_fence_before();
          }
          any = true;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->p_full[t]);
        }
        if (!ok || !(ok = wwait(&ctl->seg_full[(k + 1) % kSegments], ((k + 1) / kSegments) & 1))) break;
        __syncwarp();
        if (lane == 0) seg_done(k);
        ++k;
      }
    }
    __syncwarp();
    tc_fence_before();
    barrier_sync(1, kThreads);
    if (tid == 0 && *abort_flag) report_timeout(p.status);
  }
}

// The partial results of a row: those of its own tiles and of the nodes above its
// place, whose items were cut into pieces.  One block a (place, head): the attention
// kernel has listed where they lie (a level a lane), a thread a piece has its weight, and a warp takes
// every fourth or eighth piece, columns a lane; the warps' sums are added in order.
// 256 threads as long as all blocks are resident (28 heads x 24 places: 5 us, with
// 128 threads 6.5), 128 beyond (32 heads x 64 places: 6 us, with 256 threads 11): a chain
// of dependent loads bounds it.  An SM holds 6 blocks of 256 at d = 128 (40 registers a
// thread), 8 at d = 64 (32).  Whole steps with 256 and with 128 threads, d = 128: 900 rows 22.6 and
// 22.6 us, 1000 rows 25.4 and 23.5, 1200 rows 28.6 and 26.2; d = 64: 1200 rows 23.3 and 23.5, 1536 rows 28.1 and 26.2.
template <int D>
constexpr unsigned kWideRows = (D == 128 ? 6 : 8) * kSMs;
template <int D, int kMerge>
__global__ void __launch_bounds__(kMerge) shared_merge_kernel(const SharedParams p) {
  constexpr int L = 1 + kPlanLevels, E = D / 32, W = kMerge / 32;
  __shared__ long long s_row[L];               // a level's first partial row, of its first CTA
  __shared__ int s_second[L], s_start[L + 1];  // the second stream's distance (0: one result a piece), results in front
  __shared__ float s_red[2][W], s_w[kMerge], s_o[W][D];
  __shared__ long long s_at[kMerge];
  let_next_start();
  wait_for_previous();
  const int32_t* plan = valid_plan(p);
  const int G = p.G, i = blockIdx.x / p.Hq, h = blockIdx.x - i * p.Hq, kvh = h / G, g = h - kvh * G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = place_of(plan, i, p.B);
  if (warp == 0) {
    const int levels = plan != nullptr ? L : 1;
    Parts x{0, 0, 0};
    if (lane < levels) x = p.parts[(static_cast<long>(i) * p.Hkv + kvh) * levels + lane];
    if (length_of(p, b) == 0) x.count = 0;
    int sum = x.count;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane < L) {
      s_row[lane] = x.row + g;
      s_second[lane] = x.second;
      s_start[lane] = sum - x.count;
      if (lane == L - 1) s_start[L] = sum;
    }
  }
  __syncthreads();
  const int all = s_start[L];
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int q0 = 0; q0 < all; q0 += kMerge) {
    const int q = q0 + tid;
    long long at = -1;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (q < all) {
      int v = 0;
#pragma unroll
      for (int k = 1; k < L; ++k) v += q >= s_start[k];
      const int x = q - s_start[v], second = s_second[v];
      at = s_row[v] + static_cast<long long>(second > 0 ? x >> 1 : x) * kRows + (second > 0 && (x & 1) ? second : 0);
      if (at >= p.part_rows) at = -1;
      if (at >= 0) ml = p.part_ml[at];
      if (ml.x == -INFINITY && ml.y == 0.f) at = -1;  // (a stream that had no tile of the row's)
    }
    float top = ml.x;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    if (lane == 0) s_red[0][warp] = top;
    __syncthreads();
    float now = m;
#pragma unroll
    for (int k = 0; k < W; ++k) now = fmaxf(now, s_red[0][k]);
    // (a row of NaN has no maximum and a sum of NaN)
    const float w = at < 0 ? 0.f : ex2_approx(ml.x - now), keep = m == -INFINITY ? 1.f : ex2_approx(m - now);
    float sum = at < 0 ? 0.f : w * ml.y;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) s_red[1][warp] = sum;
    s_w[tid] = w;
    s_at[tid] = at;
    __syncthreads();
    l *= keep;
#pragma unroll
    for (int k = 0; k < W; ++k) l += s_red[1][k];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    m = now;
    const int n = min(kMerge, all - q0);
#pragma unroll 4
    for (int k = warp; k < n; k += W) {
      const long long from = s_at[k];
      if (from >= 0) {
        const float ws = s_w[k];
        const float* in = p.part_o + from * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(in);
          o[0] += ws * v.x, o[1] += ws * v.y, o[2] += ws * v.z, o[3] += ws * v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(in);
          o[0] += ws * v.x, o[1] += ws * v.y;
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  const size_t to = static_cast<size_t>(b) * p.Hq + h;
  if (tid < D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) v += s_o[k][tid];
    // (a sequence without keys: zeros; NaN stays)
    p.o[to * D + tid] = __float2bfloat16(l == 0.f ? 0.f : v / l);
  }
  // (a row without keys, or whose scores are all -infinity, adds nothing to the weights either)
  if (p.lse != nullptr && tid == 0) p.lse[to] = l == 0.f ? INFINITY : m + log2f(l);
}

// weights[b][kvh][key] += sum over the group's heads of exp2(s * scale * log2e - lse).
// A warp a tile, 4 columns a lane.
__global__ void __launch_bounds__(256) weigh_kernel(const SharedParams p) {
  wait_for_previous();
  const int b = blockIdx.z, kvh = blockIdx.y, lane = threadIdx.x & 31;
  const int len = length_of(p, b), nT = tiles_of(len);
  for (int tile = blockIdx.x * 8 + (threadIdx.x >> 5); tile < nT; tile += gridDim.x * 8) {
    const int shift = tile == nT - 1 ? nT * kTile - len : 0;
    const size_t head = static_cast<size_t>(b) * p.Hq + static_cast<size_t>(kvh) * p.G;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < p.G; ++g) {
      const float lse = p.lse[head + g];
      const float4 s =
          *reinterpret_cast<const float4*>(p.scores + ((head + g) * p.max_pages + tile) * kTile + lane * 4);
      sum.x += ex2_approx(fmaf(s.x, p.scale_log2, -lse));
      sum.y += ex2_approx(fmaf(s.y, p.scale_log2, -lse));
      sum.z += ex2_approx(fmaf(s.z, p.scale_log2, -lse));
      sum.w += ex2_approx(fmaf(s.w, p.scale_log2, -lse));
    }
    float* w = p.weights + (static_cast<size_t>(b) * p.Hkv + kvh) * p.max_pages * kTile + static_cast<size_t>(tile) * kTile;
    if (shift == 0) {
      float4* to = reinterpret_cast<float4*>(w + lane * 4);
      const float4 old = *to;
      *to = make_float4(old.x + sum.x, old.y + sum.y, old.z + sum.z, old.w + sum.w);
    } else {
      const float part[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lane * 4 + e >= shift) w[lane * 4 + e - shift] += part[e];
    }
  }
}

template <int D>
cudaError_t launch_one(const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p, cudaStream_t st) {
  auto* fn = shared_decode_kernel<D>;
  static const int launch_regs = [fn] {
    cudaFuncAttributes attr{};
    return cudaFuncGetAttributes(&attr, fn) == cudaSuccess ? attr.numRegs : -1;
  }();
  if (launch_regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), Cfg<D>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  e = launch_behind(fn, p.ctas, kThreads, Cfg<D>::kSmemBytes, st, tk, tv, p);
  if (e != cudaSuccess) return e;
  const unsigned rows = static_cast<unsigned>(p.B) * p.Hq;
  e = rows <= kWideRows<D> ? launch_behind(shared_merge_kernel<D, 256>, rows, 256, 0, st, p)
                            : launch_behind(shared_merge_kernel<D, 128>, rows, 128, 0, st, p);
  if (e != cudaSuccess || p.weights == nullptr) return e;
  const int blocks = (p.max_pages + 7) / 8;
  return launch_behind(weigh_kernel, dim3(blocks < 64 ? blocks : 64, p.Hkv, p.B), 256, 0, st, p);
}

constexpr size_t up128(size_t n) { return (n + 127) / 128 * 128; }

}  // namespace

// One CTA an SM, fewer where there cannot be work for all.
int shared_ctas(int B, int Hq, int Hkv, int max_pages) {
  const long most = static_cast<long>(B) * Hkv * max_pages;
  return static_cast<int>(most < kSMs ? most : kSMs);
}

SharedSpace shared_space(int B, int Hq, int Hkv, int max_pages, int d, bool plan, bool weights) {
  SharedSpace s{};
  // Rows of all nodes' items (a place has one node, with a plan up to kPlanLevels
  // more; twice where the streams alternate; items of few rows round up by one
  // block's remainder), and room for every CTA to begin a piece of its own.
  const long levels = plan ? 1 + kPlanLevels : 1;
  const long ctas = shared_ctas(B, Hq, Hkv, max_pages);
  s.part_rows = 2 * levels * B * static_cast<long>(Hq) + (ctas + 1) * kRows;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up128(n);
    return here;
  };
  s.part_o = take(static_cast<size_t>(s.part_rows) * d * sizeof(float));
  s.part_ml = take(static_cast<size_t>(s.part_rows) * sizeof(float2));
  s.parts = take(static_cast<size_t>(levels) * B * Hkv * sizeof(Parts));
  s.lse = weights ? take(static_cast<size_t>(B) * Hq * sizeof(float)) : 0;
  s.scores = weights ? take(static_cast<size_t>(B) * Hq * max_pages * kTile * sizeof(float)) : 0;
  s.bytes = at + 128;  // (the workspace may begin anywhere on a 16-byte boundary)
  return s;
}

cudaError_t launch_shared_decode(int d, const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p,
                                 cudaStream_t st) {
  return d == 128 ? launch_one<128>(tk, tv, p, st) : launch_one<64>(tk, tv, p, st);
}

}  // namespace ssattn

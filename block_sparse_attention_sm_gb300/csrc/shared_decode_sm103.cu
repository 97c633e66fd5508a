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
// Work: an item is (node, KV head, block of up to 256 rows), as long as the
// node has tiles.  All items' tiles laid end to end are cut into equal pieces,
// one a CTA, so that the SMs end together whatever the lengths; a piece ends at
// an item's end too.  Every piece writes its rows' (m, l, O) in fp32, and
// merge_kernel joins them.  The cuts follow from the plan and the lengths, which
// every CTA adds up for itself at its start (2 B nodes): nothing comes from the
// host, the lengths may change from step to step under the same plan.
//
// One CTA: two streams t = 0, 1, each with scores S_t, weights P_t (bf16, over
// S_t) and output O_t in TMEM (128 columns each of S and O) and a softmax
// warpgroup, one thread a row.  Of more than 128 rows each stream has half, and
// both take every tile.  Of fewer both have the same rows and take alternate
// tiles: the way of a tile from its scores to P.V is longer than the time its
// bytes take, so two are under way at once.  Scores: S_t = Q_t K^T (SS form,
// K-major, 128-byte swizzle); O_t += P_t V (TS form, V MN-major).
//
// Warps 0-3 / 4-7 softmax of stream 0 / 1 (they also load their rows of Q: the
// next piece's before they write this one's result), 8 loads K and V tiles
// through one ring, 9 issues the MMAs, 10 works out the pieces.
//
// The last tile of a sequence, of r < 128 keys, is loaded from row r - 128 of
// its page: zeros come in front, the keys follow, and what the page holds behind
// the sequence's end is never read.
//
// With weights the raw scores also go to the workspace (4 G bytes a key and KV
// head, beside 4 d of K and V), and when the merge has the row's denominator,
// weigh_kernel adds up exp2(s - lse) over the group's heads.  Each sum is made
// by one thread in the order of the heads: the same from run to run.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx_sm103.cuh"
#include "shared_decode.cuh"

namespace ssattn {

namespace {

constexpr float kRescaleLog2 = 8.0f;  // lazy-rescale slack, exp2 domain
constexpr int kSMs = 152;
constexpr int kThreads = 384;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpPlan = 10;
constexpr int kRows = 256;  // rows of an item
constexpr int kPieces = 4;  // published pieces
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
  static constexpr int kCtlBytes = 1536;
  static constexpr int kSmemBytes = kCtlOff + kCtlBytes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
};

// The tiles [t0, t1) of places [first, first + count).
struct Node {
  int first, count, t0, t1;
};

// A run of tiles of one item.
struct Piece {
  int n;          // tiles; 0: no more pieces
  int t0;         // the first of them
  int kvh;
  int first;      // the node's first place
  int row0, rows; // of the node's rows (place x head of the group)
  int both;       // each stream has half the rows and takes every tile; else all rows, alternate tiles
  int last, shift;  // a sequence's last tile, the zero rows in front of its keys (-1: none here)
  int b;          // a sequence that has these tiles
  long long out;  // its first partial row (-1: no room)
};

struct Ctl {
  uint64_t r_full[10], r_empty[10];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int n_issued;
  // the start of this CTA's share: node, its first tile and row among all
  int node;
  long long at, rows, total;
  long long scan[2][kThreads / 32];
  Piece piece[kPieces];
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

// How a node's rows are dealt to items, and an item's rows in the partial results.
struct Deal {
  int blocks, rows;   // items a KV head, rows of an item (the last may have fewer)
  int part;           // partial rows of a piece: two results each where the streams take alternate tiles
};
__device__ __forceinline__ Deal deal_of(const Node& x, int G) {
  const int all = x.count * G;
  Deal d;
  d.blocks = max(1, (all + kRows - 1) / kRows);
  d.rows = (all + d.blocks - 1) / d.blocks;
  d.part = d.rows <= kTile ? 2 * d.rows : d.rows;
  return d;
}

// Inclusive sums over the block of two values; the totals in t0, t1.
__device__ void block_sums(long long& a, long long& b, long long (*scan)[kThreads / 32], long long* ta) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += x, b += y;
  }
  if (lane == 31) scan[0][warp] = a, scan[1][warp] = b;
  __syncthreads();
  long long all = 0, pa = 0, pb = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) pa += scan[0][w], pb += scan[1][w];
    all += scan[0][w];
  }
  a += pa;
  b += pb;
  *ta = all;
}

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
  const int32_t* plan = valid_plan(p);

  if (tid == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&ctl->r_full[s], 1);
      mbar_init(&ctl->r_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ctl->q_full[t], 4);
      mbar_init(&ctl->s_full[t], 1);
      mbar_init(&ctl->p_full[t], 4);
      mbar_init(&ctl->o_full[t], 1);
      mbar_init(&ctl->o_free[t], 4);
    }
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(&ctl->piece_full[s], 1);
      mbar_init(&ctl->piece_empty[s], 10);  // softmax warps, loader, issuer
    }
    mbar_init(&ctl->mma_done, 1);
    ctl->abort_flag = 0;
    ctl->n_issued = 0;
    ctl->node = -1;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // Every node's tiles and partial rows, added up; this CTA's share begins in
  // the node that its first tile falls into.
  const int nodes = plan != nullptr ? 2 * p.B : p.B;
  {
    const int each = (nodes + kThreads - 1) / kThreads, n0 = min(nodes, tid * each), n1 = min(nodes, n0 + each);
    long long tiles = 0, rows = 0;
    for (int n = n0; n < n1; ++n) {
      const Node x = node_of(p, plan, n);
      const Deal d = deal_of(x, p.G);
      tiles += static_cast<long long>(x.t1 - x.t0) * d.blocks * p.Hkv;
      rows += static_cast<long long>(d.blocks) * p.Hkv * d.part * (x.t1 > x.t0);
    }
    long long at = tiles, row = rows, total;
    __syncthreads();
    block_sums(at, row, ctl->scan, &total);
    at -= tiles;
    row -= rows;
    const long long per = (total + gridDim.x - 1) / gridDim.x, begin = per * blockIdx.x;
    if (blockIdx.x == 0 || (begin >= at && begin < at + tiles))
      for (int n = n0; n < n1; ++n) {
        const Node x = node_of(p, plan, n);
        const Deal d = deal_of(x, p.G);
        const long long mine = static_cast<long long>(x.t1 - x.t0) * d.blocks * p.Hkv;
        if (blockIdx.x == 0) {
          p.node_at[n] = at;
          p.node_rows[n] = row;
        }
        if (begin >= at && begin < at + mine) {
          ctl->node = n;
          ctl->at = at;
          ctl->rows = row;
        }
        at += mine;
        row += static_cast<long long>(d.blocks) * p.Hkv * d.part * (x.t1 > x.t0);
      }
    if (tid == 0) ctl->total = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const long long per = (ctl->total + gridDim.x - 1) / gridDim.x;

  // Piece number k, when it has been published (a copy: the place is given back by the caller).
  auto piece_at = [&](int k, Piece* out) -> bool {
    if (!mbar_wait(&ctl->piece_full[k % kPieces], (k / kPieces) & 1, abort_flag)) return false;
    *out = ctl->piece[k % kPieces];
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == kWarpLoad) {
      // ---------------------------------------------------------- loader
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      int e = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        Piece x;
        ok = __all_sync(0xffffffffu, piece_at(k, &x));
        if (!ok || x.n == 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->piece_empty[k % kPieces]);
        // Order of use: K0 V0 K1 V1 .. where both streams take every tile,
        // K0 K1 V0 K2 V1 .. where they alternate.
        const int32_t* pages = p.table + static_cast<long>(x.b) * p.max_pages + x.t0;
        int held = 0, page[2] = {0, 0};  // 32 tiles' pages, a lane each; those of the last two keys' tiles
        int ki = 0, vi = 0;
        while (ok && vi < x.n) {
          const bool key = ki < x.n && (x.both ? ki == vi : ki <= vi + 1);
          const int u = key ? ki : vi;
          if (key) {
            if ((u & 31) == 0) held = u + lane < x.n ? pages[u + lane] : 0;
            page[1] = page[0];
            page[0] = __shfl_sync(0xffffffffu, held, u & 31);
          }
          const int at = u == ki - (key ? 0 : 1) ? page[0] : page[1];
          const int st = e % NR;
          ok = __all_sync(0xffffffffu, mbar_wait(&ctl->r_empty[st], ((e / NR) & 1) ^ 1, abort_flag));
          if (!ok) break;
          if (lane == 0) {
            const int z = at >= 0 && at < p.num_pages ? at * p.Hkv + x.kvh : p.num_pages * p.Hkv;
            const int y = x.t0 + u == x.last ? -x.shift : 0;
            mbar_arrive_expect_tx(&ctl->r_full[st], C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(sR + st * C::kTileBytes + c * 16384, key ? &tmK : &tmV, &ctl->r_full[st], c * 64, y, z);
            *reinterpret_cast<volatile int*>(&ctl->n_issued) = e + 1;
          }
          ++e;
          if (key) ++ki; else ++vi;
        }
      }
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);
        const uint32_t sQa = smem_u32(sQ), sRa = smem_u32(sR);
        uint32_t slot = 0, par = 0;            // next ring entry
        uint32_t qn[2] = {0, 0}, pn[2] = {0, 0}, on[2] = {0, 0};  // phases
        bool ok = true;
        auto next_entry = [&](uint32_t* s) -> bool {
          if (!mbar_wait(&ctl->r_full[slot], par, abort_flag)) return false;
          *s = slot;
          if (++slot == NR) slot = 0, par ^= 1;
          return true;
        };
        for (int k = 0; ok; ++k) {
          Piece x;
          ok = piece_at(k, &x);
          if (!ok || x.n == 0) break;
          mbar_arrive(&ctl->piece_empty[k % kPieces]);
          const bool both = x.both != 0;
          const int steps = both ? 2 * x.n : x.n;
          uint32_t ks = 0, vs = 0;
          for (int i = 0; ok && i < steps + 2; ++i) {
            const int t = i & 1;
            if (i >= 2) {  // P.V of step i - 2
              if ((!both || t == 0) && !(ok = next_entry(&vs))) break;
              if (i < 4) {  // the stream's first of the piece: its O has been read
                ok = mbar_wait(&ctl->o_free[t], (on[t] & 1) ^ 1, abort_flag);
                ++on[t];
                if (!ok) break;
              }
              ok = mbar_wait(&ctl->p_full[t], pn[t] & 1, abort_flag);
              ++pn[t];
              if (!ok) break;
              tc_fence_after();
              const uint64_t dv = smem_desc(sRa + vs * C::kTileBytes, 16384, 1024);
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                mma_bf16_ts(tmem + C::kColO + 128 * t, tmem + C::kColS + 128 * t + kk * 8, dv + ((kk * 2048) >> 4),
                            idO, (i >= 4 || kk > 0) ? 1u : 0u);
              if (!both || t == 1) mma_commit(&ctl->r_empty[vs]);
              if (i >= steps) mma_commit(&ctl->o_full[t]);
            }
            if (i < steps) {  // scores of step i
              if ((!both || t == 0) && !(ok = next_entry(&ks))) break;
              if (i < 2) {
                ok = mbar_wait(&ctl->q_full[t], qn[t] & 1, abort_flag);
                ++qn[t];
                if (!ok) break;
              }
              tc_fence_after();
              const uint64_t dq = smem_desc(sQa + t * C::kTileBytes, 16, 1024);
              const uint64_t dk = smem_desc(sRa + ks * C::kTileBytes, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                mma_bf16_ss(tmem + C::kColS + 128 * t, dq + off, dk + off, idS, kk > 0 ? 1u : 0u);
              }
              mma_commit(&ctl->s_full[t]);
              if (!both || t == 1) mma_commit(&ctl->r_empty[ks]);
            }
          }
        }
        mma_commit(&ctl->mma_done);
        mbar_wait(&ctl->mma_done, 0, nullptr);
      }
      __syncwarp();
    } else if (warp == kWarpPlan) {
      // ---------------------------------------------------------- pieces
      if (lane == 0) {
        long long at = per * blockIdx.x;
        const long long end = min(at + per, ctl->total);
        int n = ctl->node;
        long long node_at = ctl->at, node_rows = ctl->rows;
        for (int k = 0;; ++k) {
          Piece x{};
          if (at < end && n >= 0) {
            Node nd = node_of(p, plan, n);
            Deal d = deal_of(nd, p.G);
            int T = nd.t1 - nd.t0;
            while (n < nodes && at >= node_at + static_cast<long long>(T) * d.blocks * p.Hkv) {
              node_at += static_cast<long long>(T) * d.blocks * p.Hkv;
              node_rows += T > 0 ? static_cast<long long>(d.blocks) * p.Hkv * d.part : 0;
              if (++n == nodes) break;
              nd = node_of(p, plan, n);
              d = deal_of(nd, p.G);
              T = nd.t1 - nd.t0;
            }
            if (n < nodes) {
              const long long in = at - node_at;
              const int item = static_cast<int>(in / T), u = static_cast<int>(in - static_cast<long long>(item) * T);
              x.n = static_cast<int>(min(static_cast<long long>(T - u), end - at));
              x.t0 = nd.t0 + u;
              x.kvh = item / d.blocks;
              x.first = nd.first;
              x.row0 = (item - x.kvh * d.blocks) * d.rows;
              x.rows = min(d.rows, nd.count * p.G - x.row0);
              x.both = d.rows > kTile;
              x.b = place_of(plan, nd.first, p.B);
              x.last = -1;
              if (n < p.B) {
                const int len = length_of(p, x.b);
                x.last = len % kTile != 0 ? tiles_of(len) - 1 : -1;
                x.shift = kTile - len % kTile;
              }
              x.out = node_rows + static_cast<long long>(item) * d.part + static_cast<long long>(blockIdx.x) * kRows;
              if (x.out + d.part > p.part_rows) x.out = -1;
              at += x.n;
            }
          }
          if (!mbar_wait(&ctl->piece_empty[k % kPieces], ((k / kPieces) & 1) ^ 1, abort_flag)) break;
          ctl->piece[k % kPieces] = x;
          mbar_arrive(&ctl->piece_full[k % kPieces]);  // (release: the others read it behind their wait)
          if (x.n == 0) break;
        }
      }
      __syncwarp();
    }
    if (warp == kWarpLoad && lane == 0 && *abort_flag) {
      // let the copies in flight land before shared memory is released
      const int n = *reinterpret_cast<volatile int*>(&ctl->n_issued);
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
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t colS = lane_base + C::kColS + 128 * t, colO = lane_base + C::kColO + 128 * t;
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f32x2(sl2, sl2);
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
    };
    // Rows of this stream of piece x: [first, first + count) of the node's.
    auto my_rows = [&](const Piece& x, int* first) -> int {
      const bool both = x.both != 0;
      const int half = (x.rows + 1) / 2;
      *first = x.row0 + (both && t == 1 ? half : 0);
      return !both ? x.rows : t == 0 ? half : x.rows - half;
    };
    auto steps_of = [&](const Piece& x) { return x.both ? x.n : (x.n + 1 - t) / 2; };
    // Row i of the stream: 16-byte word j at j ^ (i & 7) of its 128-byte rows.
    auto load_q = [&](const Piece& x) {
      int first;
      const int n = my_rows(x, &first);
      constexpr int W = D / 8, RS = 128 / W;  // words of a row, rows a pass
      const int j = row % W;
      uint8_t* to = sQ + t * C::kTileBytes + (j >> 3) * 16384;
      for (int i0 = 0; i0 < n; i0 += 8 * RS) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = i0 + u * RS + row / W;
          if (i < n) {
            const int r = first + i, place = r / p.G;
            const int b = place_of(plan, x.first + place, p.B);
            v[u] = *reinterpret_cast<const uint4*>(
                p.q + b * p.q_stride + static_cast<long>(x.kvh * p.G + (r - place * p.G)) * D + j * 8);
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = i0 + u * RS + row / W;
          if (i < n) *reinterpret_cast<uint4*>(to + i * 128 + (((j & 7) ^ (i & 7)) << 4)) = v[u];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[t]);
    };
    uint32_t ns = 0, no = 0;
    Piece x;
    bool ok = __all_sync(0xffffffffu, piece_at(0, &x));
    if (ok && x.n > 0 && steps_of(x) > 0) load_q(x);
    for (int k = 0; ok && x.n > 0; ++k) {
      const int steps = steps_of(x);
      const bool both = x.both != 0;
      int first;
      const int n_rows = my_rows(x, &first);
      const bool mine = row < n_rows, warp_live = (warp & 3) * 32 < n_rows;
      float* dump = nullptr;  // this row's scores in the workspace
      if (p.scores != nullptr && mine) {
        const int r = first + row, place = r / p.G, b = place_of(plan, x.first + place, p.B);
        dump = p.scores + (static_cast<size_t>(b) * p.Hq + x.kvh * p.G + (r - place * p.G)) * p.max_pages * kTile;
      }
      float m = -INFINITY, m_used = -INFINITY, l = 0.f;
      for (int i = 0; i < steps; ++i) {
        if (!wwait(&ctl->s_full[t], ns & 1)) {
          ok = false;
          break;
        }
        ++ns;
        if (warp_live) {
          tc_fence_after();
          const int tile = x.t0 + (both ? i : 2 * i + t);
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32p(colS + 32 * c, sr + 32 * c);
          tmem_wait_ld();
          if (dump != nullptr) {
            float4* to = reinterpret_cast<float4*>(dump + static_cast<size_t>(tile) * kTile);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              to[c] = make_float4(__uint_as_float(sr[4 * c]), __uint_as_float(sr[4 * c + 1]),
                                  __uint_as_float(sr[4 * c + 2]), __uint_as_float(sr[4 * c + 3]));
          }
          if (tile == x.last) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e < x.shift) sr[e] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 64; ++e)
            mx[e & 3] = fmax3(mx[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
          m = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          float alpha = 1.f;
          bool rescale = false;
          if (m_used == -INFINITY) {
            m_used = m;  // the row's first keys
          } else if ((m - m_used) * sl2 > kRescaleLog2) {
            alpha = ex2_approx((m_used - m) * sl2);
            m_used = m;
            l *= alpha;
            rescale = true;
          }
          if (__any_sync(0xffffffffu, rescale) && i > 0) {
            // (the scores' commit covers P.V of the stream's step before)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t orr[32];
              tmem_ld32p(colO + c * 32, orr);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
              tmem_st32p(colO + c * 32, orr);
            }
          }
          // P = exp2(s * scale * log2e - m), rounded to bf16 for P.V (2^-8 of
          // a weight); l adds up the unrounded ones.
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
          tmem_st32p(colS, sr);
          tmem_st32p(colS + 32, sr + 32);
          tmem_wait_st();
          const uint64_t lsum = add_f32x2(ls[0], ls[1]);
          l += f32x2_lo(lsum) + f32x2_hi(lsum);
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[t]);
      }
      if (!ok) break;
      // The stream's score MMAs are done: its Q tile is free for the next piece.
      Piece y;
      ok = __all_sync(0xffffffffu, piece_at(k + 1, &y));
      if (!ok) break;
      if (y.n > 0 && steps_of(y) > 0) load_q(y);
      if (steps > 0) {
        ok = wwait(&ctl->o_full[t], no & 1);
        ++no;
        if (!ok) break;
      }
      if (warp_live && x.out >= 0) {
        const long long at = x.out + (first - x.row0) + row + (!both && t == 1 ? x.rows : 0);
        if (steps > 0) {
          tc_fence_after();
          float4* to = reinterpret_cast<float4*>(p.part_o + at * D);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t orr[32];
            tmem_ld32p(colO + c * 32, orr);
            tmem_wait_ld();
            if (mine)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                to[c * 8 + e] = make_float4(__uint_as_float(orr[4 * e]), __uint_as_float(orr[4 * e + 1]),
                                            __uint_as_float(orr[4 * e + 2]), __uint_as_float(orr[4 * e + 3]));
          }
        }
        if (mine) p.part_ml[at] = make_float2(m_used == -INFINITY ? -INFINITY : m_used * sl2, l);
      }
      if (steps > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_free[t]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->piece_empty[k % kPieces]);
      x = y;
    }
    __syncwarp();
    tc_fence_before();
    barrier_sync(1, kThreads);
    if (tid == 0 && *abort_flag) report_timeout(p.status);
  }
}

// The partial results of a row: along its place's node and those above it, the
// pieces that their items were cut into.  One block a (place, head); a warp
// takes every fourth result.
template <int D>
__global__ void __launch_bounds__(128) shared_merge_kernel(const SharedParams p, int ctas) {
  __shared__ float s_m[4], s_l[4];
  __shared__ float s_o[4][D];
  const int32_t* plan = valid_plan(p);
  const int i = blockIdx.x / p.Hq, h = blockIdx.x - i * p.Hq;
  const int kvh = h / p.G, g = h - kvh * p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = place_of(plan, i, p.B);
  const int nodes = plan != nullptr ? 2 * p.B : p.B;
  // all tiles, as the attention kernel counted them
  const Node end = node_of(p, plan, nodes - 1);
  const long long total =
      p.node_at[nodes - 1] + static_cast<long long>(end.t1 - end.t0) * deal_of(end, p.G).blocks * p.Hkv;
  const long long per = max(1ll, (total + ctas - 1) / ctas);
  constexpr int E = D / 32;  // entries of O a lane has
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (length_of(p, b) > 0) {
    int n = i;
    for (int level = 0; n >= 0 && n < nodes && level <= kPlanLevels; ++level) {
      const Node x = node_of(p, plan, n);
      const int T = x.t1 - x.t0, r = (i - x.first) * p.G + g;
      if (T > 0 && r >= 0 && r < x.count * p.G) {
        const Deal d = deal_of(x, p.G);
        const int blk = r / d.rows, rr = r - blk * d.rows;
        const bool both = d.rows > kTile;
        const int item = kvh * d.blocks + blk;
        const long long a = p.node_at[n] + static_cast<long long>(item) * T;
        const long long row = p.node_rows[n] + static_cast<long long>(item) * d.part + rr;
        const int c0 = static_cast<int>(a / per), c1 = static_cast<int>((a + T - 1) / per);
        const int parts = (c1 - c0 + 1) * (both ? 1 : 2);
        for (int q0 = warp; q0 < parts; q0 += 128) {  // 32 results of this warp's at a time: a lane's each
          const int q = q0 + 4 * lane;
          long long at = -1;
          float2 ml = make_float2(-INFINITY, 0.f);
          if (q < parts) {
            const int c = c0 + (both ? q : q >> 1);
            at = row + static_cast<long long>(c) * kRows + (!both && (q & 1) ? d.rows : 0);
            if (at >= p.part_rows) at = -1;
            if (at >= 0) ml = p.part_ml[at];
            if (ml.x == -INFINITY && ml.y == 0.f) at = -1;  // (a stream that had no tile)
          }
          float top = ml.x;
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
          const float now = fmaxf(m, top);
          const float keep = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2_approx(m - now);
          const float w = at < 0 ? 0.f : ex2_approx(ml.x - now);
          l *= keep;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] *= keep;
          l += w * ml.y;
          m = now;
          for (uint32_t some = __ballot_sync(0xffffffffu, at >= 0); some != 0; some &= some - 1) {
            const int s = __ffs(some) - 1;
            const float ws = __shfl_sync(0xffffffffu, w, s);
            const float* from = p.part_o + __shfl_sync(0xffffffffu, at, s) * D + lane * E;
            if constexpr (E == 4) {
              const float4 v = *reinterpret_cast<const float4*>(from);
              o[0] += ws * v.x, o[1] += ws * v.y, o[2] += ws * v.z, o[3] += ws * v.w;
            } else {
              const float2 v = *reinterpret_cast<const float2*>(from);
              o[0] += ws * v.x, o[1] += ws * v.y;
            }
          }
        }
      }
      n = plan != nullptr ? plan[kPlanHead + p.B + static_cast<long>(n) * kNodeWords + 4] : -1;
    }
  }
  // (each lane has added up its own results' sums)
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), sum = 0.f, w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[q] = s_m[q] == -INFINITY ? (s_l[q] == 0.f ? 0.f : 1.f) : ex2_approx(s_m[q] - top);
    sum += w[q] * s_l[q];
  }
  const size_t at = static_cast<size_t>(b) * p.Hq + h;
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) v += w[q] * s_o[q][threadIdx.x];
    // (a sequence without keys: zeros; NaN stays)
    p.o[at * D + threadIdx.x] = __float2bfloat16(sum == 0.f ? 0.f : v / sum);
  }
  if (p.lse != nullptr && threadIdx.x == 0) p.lse[at] = top + log2f(sum);
}

// weights[b][kvh][key] += sum over the group's heads of exp2(s * scale * log2e - lse).
// A warp a tile, 4 columns a lane.
__global__ void __launch_bounds__(256) weigh_kernel(const SharedParams p) {
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
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  fn<<<p.ctas, kThreads, Cfg<D>::kSmemBytes, st>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  shared_merge_kernel<D><<<static_cast<unsigned>(p.B) * p.Hq, 128, 0, st>>>(p, p.ctas);
  if ((e = cudaGetLastError()) != cudaSuccess || p.weights == nullptr) return e;
  const int blocks = (p.max_pages + 7) / 8;
  weigh_kernel<<<dim3(blocks < 64 ? blocks : 64, p.Hkv, p.B), 256, 0, st>>>(p);
  return cudaGetLastError();
}

constexpr size_t up16(size_t n) { return (n + 15) / 16 * 16; }

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
    at += up16(n);
    return here;
  };
  s.part_o = take(static_cast<size_t>(s.part_rows) * d * sizeof(float));
  s.part_ml = take(static_cast<size_t>(s.part_rows) * sizeof(float2));
  s.node_at = take(2 * static_cast<size_t>(B) * sizeof(long long));
  s.node_rows = take(2 * static_cast<size_t>(B) * sizeof(long long));
  s.lse = weights ? take(static_cast<size_t>(B) * Hq * sizeof(float)) : 0;
  s.scores = weights ? take(static_cast<size_t>(B) * Hq * max_pages * kTile * sizeof(float)) : 0;
  s.bytes = at;
  return s;
}

cudaError_t launch_shared_decode(int d, const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p,
                                 cudaStream_t st) {
  return d == 128 ? launch_one<128>(tk, tv, p, st) : launch_one<64>(tk, tv, p, st);
}

}  // namespace ssattn

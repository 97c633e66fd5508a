// How much attention weight each cached key receives from a step's packed new
// tokens: weights[b][kvh][key] += sum over the sequence's new tokens i and the
// G query heads h of the group of softmax_h,i[key], without the attention's
// output (a prompt, or its last window, choosing which of its keys to keep).
//
// Mathematics: the weight exp2(s - lse) needs the row's denominator first, so
// there are two passes over the scores s = q.k * scale * log2e,
//   rows:  lse = log2 sum over keys of exp2(s)   (running maximum and sum)
//   keys:  w[key] += sum over rows of exp2(s - lse)
// and no other product.  The scores are computed twice because keeping them
// would take 4 bytes a score, written and read, against 2 d operations.
//
// Both passes are one kernel.  Its fixed operand is two tiles of 128 rows (A of
// the MMAs), the other streams past it in tiles of 128 (B), and every thread
// owns a row of a fixed tile, that is a TMEM lane, and reduces along its
// columns, so no sum crosses threads.  The rows' pass fixes query rows and
// streams keys; the keys' pass fixes keys and streams query rows, whose lse are
// the columns' addends.  Rows of queries: 128 / G tokens x G heads (as in the
// chunk attention).
//
// Work: an item is (sequence, KV head, fixed pair); all items' steps laid end
// to end are cut into equal shares, one a CTA.  The steps of a causal pair are
// floors of linear functions of its number, so their sums have a closed form
// (floor_sum) and a CTA finds its share without walking a list.  An item that
// is cut leaves its parts' results in the workspace, and a small kernel joins
// them in order (results do not depend on timing).
//
// One CTA: two streams t, each with a fixed tile, two score buffers in TMEM and
// two reducing warpgroups, one for each half of the columns (with one for all columns
// the two passes of a prompt of 8K take 3% longer).  A pair of one block of rows, or of
// one tile of keys, has both streams take alternate streamed tiles against that one
// instead.  Warps 0-15 reduce (stream 0, 1, 0, 1; the second pair the second half), 16
// loads, 17 and 19 issue the MMAs of stream 0 and 1, 18 works out the pieces.
//
// Bound: a step of two tiles is ~1240 cycles of MMAs (measured without any reduction: their
// operands come from shared memory) and 1024 of exponentials; it takes ~1800 in the rows'
// pass, ~1950 in the keys' (two prompts of 8K, 32 / 8 heads of 128: 801 us together, 3.1 times
// one pass's operations at the cuBLAS rate), for the reducing warps of an SM wait, load and compute in
// step with one another.  A window of 32 tokens on long prompts is bound by its keys, read
// twice (64 us a pass for 344 MB).  Measured and not taken: issuers in turns (rows +4%, keys -4%),
// the loads of 32 columns ahead of the reduction (+20%), 512 fixed rows an item, which halves what
// is streamed (+25%), the rows' tiles in reverse for what L2 still holds (-1%).
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "key_weights.cuh"
#include "ptx_sm103.cuh"

namespace ssattn {

namespace {

constexpr int kSMs = 152;
constexpr int kThreads = 640;
constexpr int kWarpLoad = 16, kWarpMma = 17, kWarpPlan = 18, kWarpMma2 = 19;
constexpr int kHalf = kTile / 2;  // columns of a reducing warpgroup
constexpr int kPieces = 3;
constexpr int kPair = 2 * kTile;
constexpr float kSlackLog2 = 40.0f;  // how far exponentials may be above 1 (exp2 domain)
constexpr int kLaunchRegs = 96, kRegsIssue = 64, kRegsReduce = 104;
static_assert(128 * kRegsIssue + 512 * kRegsReduce == kThreads * kLaunchRegs, "register split");

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kRing = (D == 128) ? 3 : 6;  // streamed tiles
  static constexpr int kRingOff = 4 * kTileBytes;   // behind two pairs of fixed tiles
  static constexpr int kCtlOff = kRingOff + kRing * kTileBytes;
  static constexpr int kCtlBytes = (D == 128) ? 3 * 1024 : 4 * 1024;
  static constexpr int kSmemBytes = kCtlOff + kCtlBytes;  // (the base is a multiple of 1024: checked)
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// Every CTA works its share out for itself before it loads anything, with cold code: so
// 32-bit divisions where the numbers fit, and those by the tokens of a block as products.
__device__ __forceinline__ long long quotient(long long a, long long b) {  // a >= 0, b > 0
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
// floor(n / tpb), n >= 0 (`tpb_inverse` = ceil(2^64 / tpb): exact for n < 2^57).
__device__ __forceinline__ long long blocks_in(const KeyWeightsParams& p, long long n) {
  return p.tpb == 1 ? n : static_cast<long long>(__umul64hi(n, p.tpb_inverse));
}

// sum over i < n of floor((a i + b) / m), a and b below m (Euclid's steps on (a, m)).
template <typename U>
__device__ __forceinline__ long long floor_sum_of(U n, U m, U a, U b) {
  long long sum = 0;
#pragma unroll 1
  while (true) {
    const U y = a * n + b;
    if (y < m) return sum;
    n = y / m;
    b = y - n * m;
    U x = m;  // (a, m) = (m, a)
    m = a;
    a = x;
    x = a / m;
    a -= x * m;
    sum += (static_cast<long long>(n) - 1) * static_cast<long long>(n) / 2 * static_cast<long long>(x);
    x = b / m;
    b -= x * m;
    sum += static_cast<long long>(n) * static_cast<long long>(x);
  }
}
__device__ __forceinline__ long long floor_sum(long long n, int m, int a, int b) {  // a, b < m <= 256
  return n < (1 << 23) ? floor_sum_of<uint32_t>(static_cast<uint32_t>(n), m, a, b) : floor_sum_of<uint64_t>(n, m, a, b);
}

// A sequence of the step.
struct Seq {
  int n, len, off;   // new tokens, keys, keys in front of the first new token (may be negative)
  int tok0;          // first new token
  int tiles, blocks; // of keys, of query rows
  long place;        // of its first pair of row blocks
};

__device__ __forceinline__ Seq seq_of(const KeyWeightsParams& p, int b) {
  Seq s;
  s.tok0 = max(0, min(p.cu_seqlens[b], p.T));
  s.n = max(0, min(p.cu_seqlens[b + 1], p.T) - s.tok0);
  s.len = max(0, min(p.seq_lens[b], p.max_pages * kTile));
  s.off = s.len - s.n;
  s.tiles = (s.len + kTile - 1) / kTile;
  s.blocks = static_cast<int>(blocks_in(p, s.n + p.tpb - 1ll));
  s.place = blocks_in(p, s.tok0) / 2 + b;
  return s;
}

// Fixed pairs of a KV head, the steps of pair i, and the steps of all pairs below i.
template <bool ROWS>
__device__ __forceinline__ int pairs_of(const Seq& s) {
  return ROWS ? (s.blocks + 1) / 2 : (s.tiles + 1) / 2;
}
template <bool ROWS>
__device__ __forceinline__ int first_step(const KeyWeightsParams& p, const Seq& s, int i) {
  // keys: the first block of query rows that sees a key of the pair
  if (ROWS || !p.causal) return 0;
  const int x = i * kPair - s.off;  // the first token that does
  return x <= 0 ? 0 : min(s.blocks, static_cast<int>(blocks_in(p, x)));
}
template <bool ROWS>
__device__ __forceinline__ int steps_of(const KeyWeightsParams& p, const Seq& s, int i) {
  if (!ROWS) return s.blocks - first_step<ROWS>(p, s, i);
  if (!p.causal) return s.tiles;
  const long long last = static_cast<long long>(s.off) + 2ll * p.tpb * (i + 1) - 1;  // key that the pair's last token sees
  return last < 0 ? 0 : static_cast<int>(min(static_cast<long long>(s.tiles), last / kTile + 1));
}
template <bool ROWS>
__device__ long long steps_below(const KeyWeightsParams& p, const Seq& s, int i) {
  if (!p.causal) return static_cast<long long>(i) * (ROWS ? s.tiles : s.blocks);
  if (ROWS) {
    // clamp(floor((off + w (q + 1) - 1) / 128) + 1, 0, tiles): zero below q0, tiles from q1 on
    const int w = 2 * p.tpb;
    const long long c = static_cast<long long>(s.off) + w - 1;
    auto pairs_to = [&](long long x) { return x <= 0 ? 0ll : blocks_in(p, x + w - 1) / 2; };  // ceil(x / w)
    const long long q0 = pairs_to(-c), q1 = max(q0, pairs_to(static_cast<long long>(kTile) * (s.tiles - 1) - c));
    const long long n = min(static_cast<long long>(i), q1) - q0;
    long long sum = 0;
    if (n > 0) {
      const long long b = c + w * q0;
      sum = n + n * (b / kTile) + (n - 1) * n / 2 * (w / kTile) + floor_sum(n, kTile, w % kTile, static_cast<int>(b % kTile));
    }
    if (i > q1) sum += (i - q1) * s.tiles;
    return sum;
  }
  const long long k0 = s.off < 0 ? 0 : s.off / kPair + 1ll;  // first pair with a step less
  const long long n = i - k0;
  long long sum = static_cast<long long>(i) * s.blocks;
  if (n > 0) {
    const int b = static_cast<int>(k0 * kPair - s.off);  // 1 .. 256, or as far as the first tokens lie behind all keys
    const int qa = static_cast<int>(blocks_in(p, kPair)), qb = static_cast<int>(blocks_in(p, b));
    sum -= n * qb + (n - 1) * n / 2 * qa + floor_sum(n, p.tpb, kPair - qa * p.tpb, b - qb * p.tpb);
  }
  return sum;
}

// Two results (m in raw scores, l) of a row become one.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2, float sl2) {
  const float top = fmaxf(m, m2);
  // (l is 0 or NaN where m is -inf)
  l = (m == -INFINITY ? l : l * ex2_approx((m - top) * sl2)) + (m2 == -INFINITY ? l2 : l2 * ex2_approx((m2 - top) * sl2));
  m = top;
}
// -log2 of the denominator, the addend of the keys' pass; a row without keys gives -infinity, and so weights of 0.
__device__ __forceinline__ float row_addend(float m, float l, float sl2) {
  return l == 0.f ? -INFINITY : m == -INFINITY ? l : -fmaf(m, sl2, log2f(l));
}

// What an item costs besides its steps (its fixed tiles, its results), in steps: causal
// pairs at the short end are many (a CTA that had them ended 20% later than others).
constexpr int kItemCost = 2;
// Items of few steps are not cut (each belongs to the CTA whose share it begins in): that
// spares the launch that joins the parts, 3 us of ~25 on small steps.
constexpr int kWholeSteps = 16;
// Cost of all pairs below i.  Step u of pair i is at cost_below(i) + kItemCost + u, and
// belongs to the CTA whose share that lies in.
template <bool ROWS>
__device__ long long cost_below(const KeyWeightsParams& p, const Seq& s, int i) {
  if (s.tiles == 0 || s.blocks == 0) return 0;  // (no items)
  return steps_below<ROWS>(p, s, i) + static_cast<long long>(kItemCost) * i;
}

// The last of the pairs with cost_below <= in: a warp looks at 32 places at a time.
template <bool ROWS>
__device__ __forceinline__ int last_pair(const KeyWeightsParams& p, const Seq& s, int pairs, long long in) {
  int lo = 0;  // (cost_below(0) = 0 <= in)
#pragma unroll 1
  for (int n = pairs; n > 1;) {  // of [lo, lo + n)
    const int step = (n + 31) / 32, x = static_cast<int>(threadIdx.x & 31) * step;
    const uint32_t below = __ballot_sync(0xffffffffu, x < n && cost_below<ROWS>(p, s, lo + x) <= in);
    const int at = (31 - __clz(below)) * step;  // (place 0 always is)
    lo += at;
    n = min(step, n - at);
  }
  return lo;
}

// A run of steps of one item.
struct Piece {
  int n, u0, steps;  // steps; the first of them, all of the item's (n = 0: no more pieces)
  int b, kvh, pair;
  int tok0, toks;    // sequence's first token, tokens
  int len, off;
  int first;         // streamed tile of step 0 of the item
  int both;          // two fixed tiles; else both streams use the first and alternate
  long place;
};

template <int NR>
struct Ctl {
  uint64_t r_full[NR], r_empty[NR];
  uint64_t lse_empty[3][2];        // keys' pass: stream t has used the entry's lse
  uint64_t f_full[2], f_empty[2];
  uint64_t s_full[4], s_empty[4];  // [stream * 2 + buffer]
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t hand_full[2], hand_empty[2];  // a stream's second half of the columns to its first
  uint64_t cross_full;                   // alternate tiles: stream 1 to stream 0
  uint64_t mma_done[2];
  uint32_t tmem_base;
  int abort_flag;
  int r_issued, f_issued;
  int b;              // this CTA's share begins in sequence b,
  long long at, head; // with `at` of the cost in front of it and `head` a KV head
  long long total;
  Piece piece[kPieces];
  union {
    struct {
      alignas(16) float lse[3][kTile];  // the rows' lse, per ring entry % 3
      float sum[2][kTile];              // a stream's results on their way
    } keys;
    float2 rows[2][kTile];
    struct {
      float used[3 * kTile];            // (left to the copies of the lse)
      long long scan[kThreads / 32];    // the warps' sums over the batch
      float room[kTile - kThreads / 16];
      Seq seq;                          // the sequence that this CTA's share begins in
    } start;
  } hand;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

template <int D, bool ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const KeyWeightsParams p) {
  using C = Cfg<D>;
  constexpr int NR = C::kRing;
  static_assert(sizeof(Ctl<NR>) <= C::kCtlBytes, "control block overflow");
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023) != 0) {  // (no static shared memory in front of it)
    if (threadIdx.x == 0) report_timeout(p.status);
    return;
  }
  let_next_start();
  uint8_t* sF = smem;
  uint8_t* sR = smem + C::kRingOff;
  auto* ctl = reinterpret_cast<Ctl<NR>*>(smem + C::kCtlOff);
  volatile int* abort_flag = &ctl->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&ctl->r_full[s], 1);
      mbar_init(&ctl->r_empty[s], 2);  // both issuers
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->f_full[s], 1);
      mbar_init(&ctl->f_empty[s], 2);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ctl->s_full[s], 1);
      mbar_init(&ctl->s_empty[s], 8);
    }
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(&ctl->piece_full[s], 1);
      mbar_init(&ctl->piece_empty[s], 19);
    }
    for (int s = 0; s < 6; ++s) mbar_init(&ctl->lse_empty[s >> 1][s & 1], 8);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->hand_full[s], 4);
      mbar_init(&ctl->hand_empty[s], 4);
    }
    mbar_init(&ctl->cross_full, 4);
    mbar_init(&ctl->mma_done[0], 1);
    mbar_init(&ctl->mma_done[1], 1);
    ctl->abort_flag = 0;
    ctl->r_issued = ctl->f_issued = 0;
    ctl->b = -1;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  {  // every sequence's steps, added up
    long long* scan = ctl->hand.start.scan;
    const int each = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    Seq s{};
    long long head = 0;
    auto cost = [&](int b) {
      s = seq_of(p, b);
      head = cost_below<ROWS>(p, s, pairs_of<ROWS>(s));
      return head * p.Hkv;
    };
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += cost(b);
    long long at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += x;
    }
    if (lane == 31) scan[warp] = at;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += scan[w];
      total += scan[w];
    }
    at -= mine;
    const long long begin = quotient(total + gridDim.x - 1, gridDim.x) * blockIdx.x;
    if (begin >= at && begin < at + mine) {
      int b = b0;
      if (each > 1) {  // (else it is the one that has just been looked at)
        long long c = cost(b);
#pragma unroll 1
        while (begin >= at + c) {
          at += c;
          c = cost(++b);
        }
      }
      ctl->b = b;
      ctl->at = at;
      ctl->head = head;
      ctl->hand.start.seq = s;
    }
    if (tid == 0) ctl->total = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int q_rows = p.tpb * p.G;                    // rows of a block of queries
  const uint32_t q_bytes = C::kChunks * q_rows * 128;

  auto piece_at = [&](int k, Piece* out) -> bool {
    if (!mbar_wait_small(&ctl->piece_full[k % kPieces], (k / kPieces) & 1, abort_flag)) return false;
    *out = ctl->piece[k % kPieces];
    return true;
  };

  if (warp >= 16) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == kWarpLoad) {
      // ---------------------------------------------------------- loader
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
      }
      int e = 0;
      uint32_t used = 0, turn = 0;  // lse places, a bit a stream: in use, parity
      bool ok = true, waited = ROWS;
      auto load_queries = [&](uint8_t* to, uint64_t* bar, const Piece& x, int block) {
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_4d(to + c * 16384, &tmQ, bar, c * 64, 0, x.kvh, x.tok0 + block * p.tpb);
      };
      auto load_keys = [&](uint8_t* to, uint64_t* bar, const Piece& x, int page) {
        const int z = page >= 0 && page < p.num_pages ? page * p.Hkv + x.kvh : p.num_pages * p.Hkv;
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) tma_load_3d(to + c * 16384, &tmK, bar, c * 64, 0, z);
      };
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        Piece x;
        ok = __all_sync(0xffffffffu, piece_at(k, &x));
        if (!ok || x.n == 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->piece_empty[k % kPieces]);
        const int32_t* pages = p.page_table + static_cast<long>(x.b) * p.max_pages;
        const int fb = k & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_small(&ctl->f_empty[fb], ((k >> 1) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          uint8_t* to = sF + fb * 2 * C::kTileBytes;
          mbar_arrive_expect_tx(&ctl->f_full[fb], (x.both ? 2 : 1) * (ROWS ? q_bytes : C::kTileBytes));
          for (int t = 0; t < (x.both ? 2 : 1); ++t) {
            if (ROWS)
              load_queries(to + t * C::kTileBytes, &ctl->f_full[fb], x, 2 * x.pair + t);
            else
              load_keys(to + t * C::kTileBytes, &ctl->f_full[fb], x, pages[2 * x.pair + t]);
          }
          *reinterpret_cast<volatile int*>(&ctl->f_issued) = k + 1;
        }
        const float* lse_of = p.lse + (static_cast<long>(x.kvh) * p.places + x.place) * kPair;
        int held = 0;
#pragma unroll 1
        for (int i = 0; ok && i < x.n; ++i, ++e) {
          const int u = x.first + x.u0 + i;
          int page = 0;
          if (ROWS) {
            if ((i & 31) == 0) held = i + lane < x.n ? pages[u + lane] : 0;
            page = __shfl_sync(0xffffffffu, held, i & 31);
          }
          const int st = e % NR, ls = e % 3;
          ok = __all_sync(0xffffffffu, mbar_wait_small(&ctl->r_empty[st], ((e / NR) & 1) ^ 1, abort_flag));
          if (!ROWS) {  // the streams that used the place of the block's lse have done so
#pragma unroll 1
            for (int t = 0; ok && t < 2; ++t) {
              const uint32_t bit = 1u << (2 * ls + t);
              if (used & bit) {
                ok = __all_sync(0xffffffffu, mbar_wait_small(&ctl->lse_empty[ls][t], (turn & bit) != 0, abort_flag));
                turn ^= bit;
              }
              used &= ~bit;
              if (x.both || (i & 1) == t) used |= bit;
            }
          }
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&ctl->r_full[st], ROWS ? C::kTileBytes : q_bytes + kTile * sizeof(float));
            if (ROWS) {
              load_keys(sR + st * C::kTileBytes, &ctl->r_full[st], x, page);
            } else {
              load_queries(sR + st * C::kTileBytes, &ctl->r_full[st], x, u);
              // (The rows' lse.  The waits of the other warps for tiles and results are bounded, that one
              // is not: they make it too before the first that depends on it.)
              if (!waited) wait_for_previous();
              waited = true;
              bulk_load(ctl->hand.keys.lse[ls], lse_of + static_cast<long>(u) * kTile, kTile * sizeof(float), &ctl->r_full[st]);
            }
            *reinterpret_cast<volatile int*>(&ctl->r_issued) = e + 1;
          }
        }
      }
    } else if (warp == kWarpMma || warp == kWarpMma2) {
      // ---------------------------------------------------------- MMAs of stream t
      // An issuer each: one's waits and commits run beside the other's MMAs.  Both
      // pass every streamed tile in order.
      const int t = __shfl_sync(0xffffffffu, warp == kWarpMma ? 0 : 1, 0);
      constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
      const uint64_t df0 = smem_desc(smem_u32(sF), 16, 1024), dr0 = smem_desc(smem_u32(sR), 16, 1024);
      uint32_t slot = 0, par = 0, sn = 0;
      auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_small(bar, parity, abort_flag));
      };
      bool ok = true;
      if (!ROWS) wait_for_previous();  // (see the loader: no tile comes before that)
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        if (!wwait(&ctl->piece_full[k % kPieces], (k / kPieces) & 1)) break;
        const int n = __shfl_sync(0xffffffffu, ctl->piece[k % kPieces].n, 0);
        const bool both = __shfl_sync(0xffffffffu, ctl->piece[k % kPieces].both, 0) != 0;
        if (n == 0) break;
        if (elect_one()) mbar_arrive(&ctl->piece_empty[k % kPieces]);
        __syncwarp();
        ok = wwait(&ctl->f_full[k & 1], (k >> 1) & 1);
        const uint64_t df = df0 + (((k & 1) * 2 + (both ? t : 0)) * C::kTileBytes >> 4);
#pragma unroll 1
        for (int i = 0; ok && i < n; ++i) {
          if (!(ok = wwait(&ctl->r_full[slot], par))) break;
          if (both || (i & 1) == t) {
            const uint32_t buf = sn & 1;
            if (!(ok = wwait(&ctl->s_empty[2 * t + buf], ((sn >> 1) & 1) ^ 1))) break;
            ++sn;
            tc_fence_after();
            const uint64_t dr = dr0 + slot * (C::kTileBytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                mma_bf16_ss(tmem + 256 * t + 128 * buf, df + off, dr + off, idS, kk > 0 ? 1u : 0u);
              }
              mma_commit(&ctl->s_full[2 * t + buf]);
              mma_commit(&ctl->r_empty[slot]);
            }
            __syncwarp();
          } else {
            if (elect_one()) mbar_arrive(&ctl->r_empty[slot]);
            __syncwarp();
          }
          if (++slot == NR) slot = 0, par ^= 1;
        }
        if (ok && elect_one()) mma_commit(&ctl->f_empty[k & 1]);
        __syncwarp();
      }
      if (elect_one()) {
        mma_commit(&ctl->mma_done[t]);
        mbar_wait(&ctl->mma_done[t], 0, nullptr);
      }
      __syncwarp();
    } else if (warp == kWarpPlan) {
      // ---------------------------------------------------------- pieces
      const long long per = quotient(ctl->total + gridDim.x - 1, gridDim.x);
      const long long at = per * blockIdx.x, end = min(at + per, ctl->total);
      int b = at < end ? ctl->b : -1, kvh = 0, pair = 0;
      long long begin = 0;  // cost in front of the item's first step
      Seq s{};
      int pairs = 0;
      if (b >= 0) {  // the item that the share begins in
        s = ctl->hand.start.seq;
        pairs = pairs_of<ROWS>(s);
        long long in = at - ctl->at;
        kvh = static_cast<int>(quotient(in, ctl->head));
        in -= kvh * ctl->head;
        pair = last_pair<ROWS>(p, s, pairs, in);
        begin = at - in + cost_below<ROWS>(p, s, pair) + kItemCost;
      }
      if (lane == 0) {
        Split split{};
        for (int k = 0;; ++k) {
          Piece x{};
#pragma unroll 1
          while (b >= 0) {
            const int steps = steps_of<ROWS>(p, s, pair);
            if (begin - (p.whole ? kItemCost : 0) >= end) break;
            if (p.whole ? at <= begin - kItemCost && steps > 0 : at < begin + steps) {
              const int u = p.whole ? 0 : static_cast<int>(max(0ll, at - begin));
              x.n = p.whole ? steps : static_cast<int>(min(static_cast<long long>(steps), end - begin)) - u;
              x.u0 = u;
              x.steps = steps;
              x.b = b;
              x.kvh = kvh;
              x.pair = pair;
              x.tok0 = s.tok0;
              x.toks = s.n;
              x.len = s.len;
              x.off = s.off;
              x.first = first_step<ROWS>(p, s, pair);
              x.both = ROWS ? 2 * pair + 1 < s.blocks : 2 * pair + 1 < s.tiles;
              x.place = s.place;
              if (u == 0 && x.n < steps) split = Split{1, b, kvh, pair, steps - x.n, static_cast<int>(min(per, 0x7fffffffll))};
            }
            // on to the next item
            begin += steps + kItemCost;
            if (++pair >= pairs) {
              pair = 0;
              if (++kvh == p.Hkv) {
                kvh = 0;
                do {
                  if (++b >= p.B) break;
                  s = seq_of(p, b);
                  pairs = pairs_of<ROWS>(s);
                } while (s.tiles == 0 || s.blocks == 0);
                if (b >= p.B) b = -1;
              }
            }
            if (x.n > 0) break;
          }
          // (A place is free when its piece is done, on the longest caches after millions of steps
          // of 1-2 us: 60 us of limit for each.  The other warps' waits end with a tile and set
          // the flag if they do not.)
          if (!ROWS && k == kPieces) wait_for_previous();
          const uint32_t more = k < kPieces ? 0u : 16u * static_cast<uint32_t>(min(ctl->piece[k % kPieces].n, 1 << 26));
          if (!mbar_wait_small(&ctl->piece_empty[k % kPieces], ((k / kPieces) & 1) ^ 1, abort_flag, kSmallTries + more)) break;
          ctl->piece[k % kPieces] = x;
          mbar_arrive(&ctl->piece_full[k % kPieces]);
          if (x.n == 0) break;
        }
        if (!ROWS) wait_for_previous();  // (which reads its own; and no CTA ends before that kernel)
        p.split[blockIdx.x] = split;
      }
      __syncwarp();
    }
    if (warp == kWarpLoad && lane == 0 && *abort_flag) {
      // let the copies in flight land before shared memory is released
      const int n = *reinterpret_cast<volatile int*>(&ctl->r_issued);
      const int f = *reinterpret_cast<volatile int*>(&ctl->f_issued);
      for (int q = 0; q < NR; ++q)
        if (n > q) mbar_wait(&ctl->r_full[q], ((n - 1 - q) / NR) & 1, nullptr);
      for (int q = 0; q < 2; ++q)
        if (f > q) mbar_wait(&ctl->f_full[q], ((f - 1 - q) / 2) & 1, nullptr);
    }
    __syncwarp();
    tc_fence_before();
    barrier_sync(1, kThreads);
    if (warp == kWarpMma) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  } else {
    // ---------------------------------------------------------- reduction of stream t, half h of its columns
    setmaxnreg_inc<kRegsReduce>();
    const int t = (warp >> 2) & 1, h = warp >> 3, row = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * t + kHalf * h;
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f32x2(sl2, sl2);
    const float slack = kSlackLog2 / sl2;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_small(bar, parity, abort_flag));
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    uint32_t sn = 0, hn = 0, cn = 0;
    int e0 = 0;  // ring entries of the pieces before
    bool ok = true;
    if (!ROWS) wait_for_previous();  // (see the loader: no score comes before that)
#pragma unroll 1
    for (int k = 0; ok; ++k, ++hn) {
      ok = wwait(&ctl->piece_full[k % kPieces], (k / kPieces) & 1);
      const Piece& x = ctl->piece[k % kPieces];
      const int n = x.n;
      if (!ok || n == 0) break;
      const bool alone = !x.both;
      // (keys: a pair of one tile has the second stream take alternate blocks of rows as well)
      const int ft = alone ? 0 : t;                       // this stream's fixed tile
      float m_used = -INFINITY, limit = -INFINITY, base = 0.f, l = 0.f;  // rows
      float sum[2] = {0.f, 0.f};                          // keys
      // rows: this thread's token and the last key that it sees; keys: this thread's key
      const int token = (2 * x.pair + ft) * p.tpb + row / p.G;
      const bool row_live = ROWS && row < q_rows && token < x.toks;
      const int lim = !row_live ? -1 : p.causal ? min(x.len - 1, x.off + token) : x.len - 1;
      const int key = (2 * x.pair + ft) * kTile + row;
      const int u0 = x.first + x.u0, toks = x.toks, ahead = key - x.off;  // keys: the first token that sees the key
      // Streamed tiles [whole_from, whole_to) count as a whole for all of the warp.
      int whole_from = 0, whole_to;
      if (ROWS) {
        whole_to = static_cast<int>(max(0ll, __reduce_min_sync(0xffffffffu, lim) + 1ll - kHalf * h + kHalf) / kTile);
      } else {
        whole_to = q_rows < kTile ? 0 : toks / p.tpb;
        if (p.causal) {  // from the first block whose token of column kHalf h sees the warp's last key
          const long long last = static_cast<long long>(key | 31) - x.off - kHalf * h / p.G;
          whole_from = last <= 0 ? 0 : static_cast<int>((last + p.tpb - 1) / p.tpb);
        }
      }
#pragma unroll 1
      for (int i = alone ? t : 0; i < n; i += alone ? 2 : 1) {
        const uint32_t buf = sn & 1;
        if (!wwait(&ctl->s_full[2 * t + buf], (sn >> 1) & 1)) {
          ok = false;
          break;
        }
        ++sn;
        tc_fence_after();
        uint32_t sr[kHalf];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32p(lane_base + 128 * buf + 32 * c, sr + 32 * c);
        tmem_wait_ld();
        tc_fence_before();
        arrive(&ctl->s_empty[2 * t + buf]);
        const int u = u0 + i;
        if (ROWS) {
          if (u >= whole_to) {
            const int vis = lim - u * kTile - kHalf * h;  // last visible column
#pragma unroll
            for (int e = 0; e < kHalf; ++e)
              if (e > vis) sr[e] = __float_as_uint(-INFINITY);
          }
          // The reference m_used is the maximum of the row's first tile as long as no
          // score is above it by more than 2^kSlackLog2 (`limit`): the maximum is formed beside
          // the exponentials, and only a row's first tile takes a second turn.
#pragma unroll 1
          while (true) {
            uint64_t ls[2] = {0ull, 0ull};
            float mx[2] = {-INFINITY, -INFINITY};
            const uint64_t base2 = f32x2(base, base);
#pragma unroll
            for (int c = 0; c < kHalf / 2; ++c) {
              const float s0 = __uint_as_float(sr[2 * c]), s1 = __uint_as_float(sr[2 * c + 1]);
              mx[c & 1] = fmax3(mx[c & 1], s0, s1);
              const uint64_t xp = fma_f32x2(f32x2(s0, s1), sl2x2, base2);
              ls[c & 1] = add_f32x2(ls[c & 1], f32x2(ex2_approx(f32x2_lo(xp)), ex2_approx(f32x2_hi(xp))));
            }
            const float top = fmaxf(mx[0], mx[1]);
            if (!__any_sync(0xffffffffu, top > limit)) {
              const uint64_t s2 = add_f32x2(ls[0], ls[1]);
              l += f32x2_lo(s2) + f32x2_hi(s2);
              break;
            }
            if (top > limit) {  // (then it is not above the new one)
              if (m_used != -INFINITY) l *= ex2_approx((m_used - top) * sl2);
              m_used = top;
              limit = top + slack;
              base = -top * sl2;
            }
          }
        } else {
          // columns: rows of block u of the queries; those that count and see the key are [lo, hi)
          const int ls_at = (e0 + i) % 3;
          const float4* lse4 = reinterpret_cast<const float4*>(ctl->hand.keys.lse[ls_at] + kHalf * h);
          uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
          // (a row that does not count may hold anything: its weight is dropped, not its score)
          auto add_up = [&](auto masked, int lo, int hi) {
#pragma unroll
            for (int c = 0; c < kHalf / 4; ++c) {
              const float4 a = lse4[c];
              const uint64_t x0 = fma_f32x2(f32x2(__uint_as_float(sr[4 * c]), __uint_as_float(sr[4 * c + 1])), sl2x2,
                                            f32x2(a.x, a.y));
              const uint64_t x1 = fma_f32x2(f32x2(__uint_as_float(sr[4 * c + 2]), __uint_as_float(sr[4 * c + 3])),
                                            sl2x2, f32x2(a.z, a.w));
              float w[4] = {ex2_approx(f32x2_lo(x0)), ex2_approx(f32x2_hi(x0)), ex2_approx(f32x2_lo(x1)),
                            ex2_approx(f32x2_hi(x1))};
              if (masked()) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (4 * c + e < lo || 4 * c + e >= hi) w[e] = 0.f;
              }
              ls[c & 1] = add_f32x2(ls[c & 1], f32x2(w[0], w[1]));
              ls[2 + (c & 1)] = add_f32x2(ls[2 + (c & 1)], f32x2(w[2], w[3]));
            }
          };
          if (u >= whole_from && u < whole_to) {
            add_up([] { return false; }, 0, kHalf);
          } else {
            const int i0 = u * p.tpb;
            const long long unseen = p.causal ? (static_cast<long long>(ahead) - i0) * p.G : 0;
            add_up([] { return true; }, static_cast<int>(max(0ll, min(static_cast<long long>(kTile), unseen))) - kHalf * h,
                   min(q_rows, (toks - i0) * p.G) - kHalf * h);
          }
          arrive(&ctl->lse_empty[ls_at][t]);
          const uint64_t s2 = add_f32x2(add_f32x2(ls[0], ls[1]), add_f32x2(ls[2], ls[3]));
          sum[0] += f32x2_lo(s2);
          sum[1] += f32x2_hi(s2);
        }
      }
      if (!ok) break;
      e0 += n;
      // The item's result, or a part of it: the second half's to the first, where the
      // streams alternate stream 1's to stream 0 (through the same place).
      float total = sum[0] + sum[1];
      auto put = [&] {
        if (ROWS) ctl->hand.rows[t][row] = make_float2(m_used, l);
        else ctl->hand.keys.sum[t][row] = total;
      };
      auto add = [&](int from) {
        if (ROWS) {
          const float2 other = ctl->hand.rows[from][row];
          join(m_used, l, other.x, other.y, sl2);
        } else {
          total += ctl->hand.keys.sum[from][row];
        }
      };
      if (h == 1) {
        if (!(ok = wwait(&ctl->hand_empty[t], (hn & 1) ^ 1))) break;
        put();
        arrive(&ctl->hand_full[t]);
      } else {
        if (!(ok = wwait(&ctl->hand_full[t], hn & 1))) break;
        add(t);
        if (alone && t == 1) {
          put();
          arrive(&ctl->cross_full);
        } else {
          arrive(&ctl->hand_empty[t]);
        }
        if (alone && t == 0) {
          if (!(ok = wwait(&ctl->cross_full, cn & 1))) break;
          ++cn;
          add(1);
          arrive(&ctl->hand_empty[1]);
        }
        if (!(alone && t == 1)) {
          const bool whole = n == x.steps;
          const long part = (2l * blockIdx.x + (x.u0 == 0 ? 1 : 0)) * kPair + ft * kTile + row;
          if (ROWS) {
            if (row_live) {
              if (whole)
                p.lse[(static_cast<long>(x.kvh) * p.places + x.place + x.pair) * kPair + ft * kTile + row] =
                    row_addend(m_used, l, sl2);
              else
                p.part_ml[part] = make_float2(m_used, l);
            }
          } else if (key < x.len) {
            if (whole)
              // (one thread adds to a cell: the same as reading, adding and writing, without waiting)
              atomicAdd(p.weights + (static_cast<long>(x.b) * p.Hkv + x.kvh) * p.max_pages * kTile + key, total);
            else
              p.part_w[part] = total;
          }
        }
      }
      arrive(&ctl->piece_empty[k % kPieces]);
    }
    __syncwarp();
    tc_fence_before();
    barrier_sync(1, kThreads);
    if (tid == 0 && *abort_flag) report_timeout(p.status);
  }
}

// Block c: the item that CTA c began and others went on with.
template <bool ROWS>
__global__ void __launch_bounds__(kPair) join_kernel(const KeyWeightsParams p) {
  let_next_start();
  wait_for_previous();
  const Split x = p.split[blockIdx.x];
  if (!x.valid) return;
  const Seq s = seq_of(p, x.b);
  const int t = threadIdx.x >> 7, row = threadIdx.x & 127;
  long at = (2l * blockIdx.x + 1) * kPair + threadIdx.x;
  if (ROWS) {
    if (row >= p.tpb * p.G || (2 * x.pair + t) * p.tpb + row / p.G >= s.n) return;
    float m = p.part_ml[at].x, l = p.part_ml[at].y;
    int c = blockIdx.x + 1;
    for (int left = x.left; left > 0 && c < p.ctas; left -= x.per, ++c) {
      const float2 o = p.part_ml[2l * c * kPair + threadIdx.x];
      join(m, l, o.x, o.y, p.scale_log2);
    }
    p.lse[(static_cast<long>(x.kvh) * p.places + s.place + x.pair) * kPair + threadIdx.x] = row_addend(m, l, p.scale_log2);
  } else {
    const int key = 2 * x.pair * kTile + threadIdx.x;
    if (key >= s.len) return;
    float sum = p.part_w[at];
    int c = blockIdx.x + 1;
    for (int left = x.left; left > 0 && c < p.ctas; left -= x.per, ++c) sum += p.part_w[2l * c * kPair + threadIdx.x];
    p.weights[(static_cast<long>(x.b) * p.Hkv + x.kvh) * p.max_pages * kTile + key] += sum;
  }
}

template <int D, bool ROWS>
cudaError_t launch_pass(const CUtensorMap& tq, const CUtensorMap& tk, const KeyWeightsParams& p, cudaStream_t st) {
  auto* fn = key_weights_kernel<D, ROWS>;
  static const int launch_regs = [fn] {
    cudaFuncAttributes attr{};
    return cudaFuncGetAttributes(&attr, fn) == cudaSuccess ? attr.numRegs : -1;
  }();
  if (launch_regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), Cfg<D>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  if (ROWS) {
    fn<<<p.ctas, kThreads, Cfg<D>::kSmemBytes, st>>>(tq, tk, p);
    e = cudaGetLastError();
  } else {
    e = launch_behind(fn, p.ctas, kThreads, Cfg<D>::kSmemBytes, st, tq, tk, p);
  }
  return e != cudaSuccess || p.whole ? e : launch_behind(join_kernel<ROWS>, p.ctas, kPair, 0, st, p);
}

constexpr size_t up16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

KeyWeightsSpace key_weights_space(int T, int B, int Hq, int Hkv) {
  KeyWeightsSpace s{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up16(n);
    return here;
  };
  s.lse = take(static_cast<size_t>(Hkv) * key_weights_places(T, B, kTile / (Hq / Hkv)) * kPair * sizeof(float));
  s.part_ml = take(2 * kSMs * kPair * sizeof(float2));
  s.part_w = take(2 * kSMs * kPair * sizeof(float));
  s.split = take(kSMs * sizeof(Split));
  s.bytes = at;
  return s;
}

cudaError_t launch_key_weights(int d, const CUtensorMap& tq, const CUtensorMap& tk, const KeyWeightsParams& p0,
                               cudaStream_t st) {
  KeyWeightsParams p = p0;
  p.ctas = kSMs;
  p.whole = p.max_pages <= kWholeSteps;  // (tiles of keys that a pair of row blocks sees)
  cudaError_t e = d == 128 ? launch_pass<128, true>(tq, tk, p, st) : launch_pass<64, true>(tq, tk, p, st);
  if (e != cudaSuccess) return e;
  p.whole = (p.T + p.tpb - 1) / p.tpb <= kWholeSteps;  // (row blocks that see a pair of tiles)
  return d == 128 ? launch_pass<128, false>(tq, tk, p, st) : launch_pass<64, false>(tq, tk, p, st);
}

}  // namespace ssattn

// Attention of a chunk of new tokens over the paged key/value cache, with the
// skip test, for sm_103a: chunked prefill, the verification of drafted tokens,
// mixed batches of both, and (not causal) cross attention to cached states.
//
// Mathematics: the one-pass online softmax over 128-key tiles with the skip
// vote ("Skip-Softmax" design doc, Sec. The online-softmax pass and The skip test),
// per sequence b over its L_b cached keys.  New token i of the sequence's n_b
// sees the keys up to L_b - n_b + i (causal) or all L_b.
//
// Rows: the G = Hq / Hkv query heads of a KV head share its keys, so a row
// block packs 128 / G tokens x G heads as the 128 rows of an MMA (row = token *
// G + head): a few drafted tokens of a group fill a block that G separate
// heads would leave mostly empty, K and V are read once for the group, and a
// causal block's diagonal is 128 / G tokens wide instead of 128.
//
// A page is one tile, reached through the page table; K and V tiles are TMA
// boxes of the pool seen as [pages * Hkv][128][d].  The last tile of a
// sequence, of r < 128 keys, is loaded from row r - 128: the box's first
// 128 - r rows lie before the page and are filled with zeros, the keys follow,
// and what the page holds behind the sequence's end is never read (it may be
// NaN, which zero weights would not remove from P V).  Scores of the leading
// columns are masked.
//
// Machinery (that of the CTA-pair prefill kernel): a cluster of two CTAs takes
// two row blocks and shares every tile through two-SM MMAs (cta_group::2, M =
// 256); each SM stages half of each K and V tile.  TMEM per SM: three score
// buffers and O.  Two softmax warpgroups per CTA take alternate tiles, one
// thread per row, and hand the rows' running maximum on through shared memory;
// P goes back to TMEM as bf16 (P <= 2^8 relative to the reference maximum;
// rounded by 2^-8 of a weight at most, the sums l are of the unrounded fp32)
// and P.V accumulates in fp32.  Every wait is bounded.
//
// Units and clusters: a unit is (pair of row blocks, KV head, part of the
// tiles).  Serving batches have many short units (a decoded token over a few
// pages next to pieces of prompts), so a cluster stays resident and takes unit
// after unit: it cancels a cluster of the grid that has not been launched yet
// and does that one's unit (cluster launch control: the hardware hands them
// out as clusters become free, in no memory of ours).  Barriers, TMEM and the
// K / V rings live on: the producers load the next unit's first tiles, and the
// score issuer starts on them, while the softmax of the last unit's tail and
// its epilogue run.
//
// Roles (384 threads in each CTA): warps 0-7 softmax and vote, two warpgroups;
// warp 8 units, Q and K (it asks for the next unit when it issues the last
// loads of one; the answer comes to both CTAs, and warp 8 of each works out the
// unit's geometry and publishes it to the CTA's other warps); warp 9 V; warp 10
// of CTA 0 the score MMAs; warp 11 of CTA 0 the P.V MMAs.  With the vote warp 8
// loads V too and warp 9 of CTA 0 issues every other tile's scores.
//
// Few rows and a long cache: the tiles are dealt to parts whose states (m, l,
// O) a second kernel merges in fp32.  The ranges of the vote (num_kv_splits:
// each starts without a running maximum, so its first tile is kept) are a
// matter of the definition, not of the launch: one unit passes through several
// ranges in turn, restarting the vote's maximum, and only as many parts are
// made as there are idle clusters for (chunk_parts).
//
// d = 64 runs with value tiles padded to 128 columns (the second SM's half of
// a value tile is an out-of-range box).
//
// What bounds it (measured on GB300; 4 x 2048 new tokens over 32K keys, 32 / 8
// heads of 128).  Dense: 2.86 ms, 1490 TFLOP/s, 77% of the cuBLAS rate; the
// P.V issuer is busy throughout (8 two-SM MMAs take ~900 cycles beside the
// other issuer's, and ~500 go to barriers and commits).  With the skip test at
// ~88% skipped tiles: 1.94 ms; a tile's scores pass through MMA, commit, load,
// vote and two barriers (~2900 cycles) and TMEM holds three of them.  Short
// units: ~3 us each beside their tiles (608 units of 16 tiles: 139 us, 4.6
// TB/s).  Instructions matter: a unit's code runs out of the instruction cache,
// which is why the halves of a tile are rolled loops, what a sequence's units
// share is read from shared memory, and the issuers' paths are short.  Tried
// and slower: scores in registers with separate P buffers (two score buffers,
// 2.67 ms with the skip test); P of skipped blocks left out by a lane mask
// instead of zeros (the masked MMA form costs 8%); polling instead of
// suspended waits (2.27 ms).
#include <cuda_bf16.h>

#include "chunk_paged.cuh"
#include "common.cuh"
#include "ptx_pair_sm103.cuh"
#include "ptx_sm103.cuh"

namespace ssattn {

namespace {

constexpr float kRescaleLog2 = 8.0f;  // lazy-rescale slack (exp2 domain)
constexpr int kSoftWarps = 8;                 // two warpgroups of 4: alternate tiles
constexpr int kGroupWarps = 4;                // one thread per query row
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kThreads = kSoftThreads + 128;  // + producers and issuers
// Register split: launched at 168 per thread (384 x 168 = 64512), raised for
// the softmax warpgroups and lowered for the producers and issuers.
constexpr int kLaunchRegs = 168;
template <Mode MODE>
constexpr int kRegsDown = (MODE == Mode::kDense) ? 104 : 88;
template <Mode MODE>
constexpr int kRegsUp = (kThreads * kLaunchRegs - 128 * kRegsDown<MODE>) / 256;
static_assert(kRegsUp<Mode::kDense> == 200 && kRegsUp<Mode::kSparse> == 208, "register split");
constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10, kWarpPV = 11;
constexpr int kNB = 3;  // score buffers
constexpr int kAllKeys = 0x7ffffe00;  // a row sees every key (room for + a block's tokens)
constexpr int kSeqs = 512;  // sequences whose offsets and lengths are kept in shared memory
constexpr uint32_t kFlagKept = 1u, kFlagRescale = 2u;

// Scheduling fence for registers: the 8 values `done` are complete before,
// and the 16 values `next` are read only after, this point (a compiler hint
// that bounds how far exponentials are hoisted ahead, and so the registers
// they hold; no instruction is emitted).
__device__ __forceinline__ void order_after(uint32_t* done, uint32_t* next) {
  asm volatile(""
               : "+r"(done[0]), "+r"(done[1]), "+r"(done[2]), "+r"(done[3]), "+r"(done[4]),
                 "+r"(done[5]), "+r"(done[6]), "+r"(done[7]), "+r"(next[0]), "+r"(next[1]),
                 "+r"(next[2]), "+r"(next[3]), "+r"(next[4]), "+r"(next[5]), "+r"(next[6]),
                 "+r"(next[7]), "+r"(next[8]), "+r"(next[9]), "+r"(next[10]), "+r"(next[11]),
                 "+r"(next[12]), "+r"(next[13]), "+r"(next[14]), "+r"(next[15]));
}

// A place in a ring of N slots and the parity of its current use, STEP places
// a time (the issuers' indices: their instructions between MMAs are time the
// tensor pipe idles).
template <int N, int STEP>
struct Ring {
  uint32_t at, par;
  __device__ explicit Ring(uint32_t first, uint32_t parity = 0) : at(first), par(parity) {}
  __device__ __forceinline__ void next() {
    at += STEP;
    if (at >= N) at -= N, par ^= 1;
  }
};

template <int DQK, int DV>
struct PairCfg {
  static_assert(DQK == 64 || DQK == 128, "key width");
  static_assert(DV == 128, "value width: O occupies TMEM columns 384..511");
  static constexpr int kChunksQ = DQK / 64;             // 128-byte swizzle chunks per row
  static constexpr int kQBytes = kTile * DQK * 2;        // room of this CTA's row block
  static constexpr int kKHalfBytes = 64 * DQK * 2;      // 64 keys of a tile
  static constexpr int kKChunk = 64 * 128;               // one 64-column chunk of 64 keys
  static constexpr int kVHalfBytes = kTile * 64 * 2;    // 64 value columns of a tile
  static constexpr int kNK = 4;                          // K ring slots
  static constexpr int kNV = 5;                          // V ring slots
  static constexpr int kQOff = 0;                        // two row blocks: this unit's, the next one's
  static constexpr int kKOff = kQOff + 2 * kQBytes;
  static constexpr int kVOff = kKOff + kNK * kKHalfBytes;
  static constexpr int kCtlOff = kVOff + kNV * kVHalfBytes;
  static constexpr int kCtlBytes = 15360;
  static constexpr int kSmemBytes = kCtlOff + kCtlBytes + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColO = 384;
  static constexpr uint32_t kTmemCols = 512;
};

// A unit as the warps of one CTA need it.
struct Unit {
  int b, kvh, part;           // sequence, KV head, part of the tiles
  int j0, j1;                 // tiles of the part, of all the sequence's
  int n_pair, n_mine;         // of them, seen by either block / by this CTA's block
  int tok, toks;              // this block's first new token (of the batch), its tokens
  int lim0;                   // last key that the first of them sees (causal), or any
  int last, last_shift;       // the sequence's last tile; zero rows in front of its keys
  int range;                  // tiles of a range of the vote
  float thr_raw;              // skip iff tile_max - m < thr_raw
  int id;                     // place * 2 + CTA rank, with the KV head; -1: no more units
};

template <int NK, int NV>
struct PairCtl {
  uint64_t q_full[2];          // leader: both Q blocks landed
  uint64_t q_empty[2];         // each CTA: the unit's score MMAs are done, Q may be refilled
  uint64_t k_full[NK];         // leader: both K halves of a ring entry landed
  uint64_t v_full[NV];         // leader: both V halves landed
  uint64_t k_empty[NK];        // each CTA: its K slot may be refilled
  uint64_t v_empty[NV];        // each CTA: its V slot may be refilled
  uint64_t s_full[6];          // each CTA, per tile % kSlots: the tile's scores are in TMEM
  uint64_t dec[kNB];           // leader: both CTAs' 4 warps on the buffer's tile have decided
                               // it (CTA 0's by arrivals, CTA 1's as 16 bytes of stores)
  uint64_t drain[kSoftWarps];  // each CTA, per softmax warp: the P.V MMAs issued so far are done
  uint64_t rescaled[2][kSoftWarps];  // leader: (CTA, warp) has rescaled its part of O
  uint64_t s_free[6];          // leader, per tile % kSlots: the tile's P.V is issued (or not needed)
  uint64_t o_full;             // each CTA: the unit's last P.V is done
  uint64_t o_free;             // leader: the unit's O has been read (4 warps of each CTA)
  uint64_t handed[4];          // each CTA, per tile % 4: the rows' state after the tile is in `hand`
  uint64_t summed[4];          // each CTA, per unit % 4: the other warpgroup's share is in `fin`
  uint64_t mma_done[3];        // leader: teardown, per issuer
  uint64_t unit_full[2];       // each CTA: a unit's geometry is published
  uint64_t unit_empty[2];      // each CTA: its other warps have read it
  uint64_t next_full[2];       // each CTA: the answer to the request for a unit
  uint64_t next_empty[2];      // leader: both CTAs have read it
  alignas(16) uint32_t answer[2][4];                  // cluster launch control's
  alignas(16) uint32_t flags[kNB][kGroupWarps];       // leader: per buffer and warp of the
                                                      // tile's warpgroup, kFlagKept | kFlagRescale
  alignas(16) uint32_t peer_flags[kNB][kGroupWarps];  // leader: the same for CTA 1's warps
  uint32_t o_note[kGroupWarps];  // leader: written by CTA 1's warps to complete bytes on o_free
  uint32_t tmem_base;
  int abort_flag;
  Unit unit[2];
  uint32_t skipped[4];         // per unit % 4: tiles that the warpgroup without the last tile skipped
  float red[2][kGroupWarps];   // per warpgroup and warp: largest vote statistic of a tile
  float2 hand[4][kTile];       // per tile % 4 and row: (m, m_ref) after the tile
  float2 fin[4][kTile];        // per unit % 4 and row: (m_ref, l) of the warpgroup without the last tile
  int cu[kSeqs + 1], len[kSeqs];  // the batch's offsets and lengths (B <= kSeqs)
};

// 4-D tiled TMA load of a row block: (d, head of the group, KV head, token).
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster_addr, int c0, int c1, int c2,
                                                 int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// The sequence whose pairs include place `slot`: the last b with floor(cu[b] /
// pair) + b <= slot, 32 candidates a step.  Executed by whole warps.
__device__ __forceinline__ int sequence_of_slot(const int* cu, int B, int pair, int slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (true) {
    const int stride = (n + 31) / 32, b = lo + lane * stride;
    const int c = __popc(__ballot_sync(0xffffffffu, b < lo + n && cu[b] / pair + b <= slot));
    const int end = lo + n;
    lo += max(0, c - 1) * stride;
    if (stride == 1) return lo;
    n = min(stride, end - lo);
  }
}

// Cluster launch control: ask the hardware for a cluster of this grid that has
// not been launched.  The answer (16 bytes) lands in the shared memory of both
// CTAs and completes 16 bytes on the barrier of each.
__device__ __forceinline__ void request_cluster(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all"
      ".b128 [%0], [%1];" ::"r"(
          smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// First block of the cluster that was handed over, or -1.
__device__ __forceinline__ int requested_block(const void* answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

// DVO: the value (and output) width in memory.  DVO = 64 runs as DV = 128
// with the second SM's half of every value tile a fully out-of-range TMA box
// (read as zeros): O's columns 64.. stay zero and are not written.
template <int DQK, int DV, int DVO, Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const ChunkParams p) {
  using C = PairCfg<DQK, DV>;
  static_assert(DVO == DV || (DVO == 64 && DV == 128), "value width");
  constexpr int NK = C::kNK, NV = C::kNV;
  using Ctl = PairCtl<NK, NV>;
  static_assert(sizeof(Ctl) <= C::kCtlBytes, "control block overflow");
  constexpr bool kVote = (MODE != Mode::kDense);
  constexpr bool kTwo = kVote;  // two score issuers, one producer
  // Slots of a tile's barriers: with two issuers a slot belongs to one of them
  // (and to one softmax warpgroup), so that no waiter misses a phase of it.
  constexpr uint32_t kSlots = kTwo ? 6 : kNB;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem + C::kQOff;
  uint8_t* sK = smem + C::kKOff;
  uint8_t* sV = smem + C::kVOff;
  auto* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  volatile int* abort_flag = &ctl->abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = (rank == 0);
  const uint32_t peer_abort = map_shared(smem_u32(&ctl->abort_flag), rank ^ 1u);
  // shared::cluster address of a barrier of the leader
  auto lead = [&](uint64_t* bar) { return map_shared(smem_u32(bar), 0u); };

  // The geometry of unit number x (a whole warp; every lane returns it).
  // Later pairs of a sequence (with a causal mask: the longer) come first.
  const int* cu = p.B <= kSeqs ? ctl->cu : p.cu_seqlens;
  const int* lens = p.B <= kSeqs ? ctl->len : p.seq_lens;
  auto geometry = [&](int x) -> Unit {
    Unit u;
    const int sk = x / p.slots;  // part * Hkv + KV head
    const int slot = p.slots - 1 - (x - sk * p.slots);
    u.part = sk / p.Hkv;
    u.kvh = sk - u.part * p.Hkv;
    u.id = (u.kvh * p.slots + slot) * 2 + static_cast<int>(rank);
    const int b = sequence_of_slot(cu, p.B, 2 * p.tpb, slot);
    u.b = b;
    const int tok0 = max(0, min(cu[b], p.T));  // the sequence's new tokens
    const int n_new = max(0, min(cu[b + 1], p.T) - tok0);
    const int len = max(0, min(lens[b], p.max_pages * kTile));
    const int pr = slot - (tok0 / (2 * p.tpb) + b);
    const int off = len - n_new;  // (causal) new token i sees keys up to off + i
    const int nT = (len + kTile - 1) / kTile;
    u.last = nT - 1;
    u.last_shift = nT * kTile - len;
    u.range = max(1, (nT + p.S - 1) / p.S);
    // a part: whole ranges where there is a vote, otherwise an even share
    const int granule = kVote ? u.range : 1, n_granules = (nT + granule - 1) / granule;
    const int per = (n_granules + p.parts - 1) / p.parts * granule;
    u.j0 = min(nT, u.part * per);
    u.j1 = min(nT, u.j0 + per);
    u.thr_raw = (p.lambda_a > 0.f && len > 0)  // lambda_b = min(1, a / L_b)
                    ? logf(fminf(1.f, p.lambda_a / static_cast<float>(len))) / p.scale
                    : -INFINITY;
    u.n_pair = u.n_mine = u.toks = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int i0 = (2 * pr + t) * p.tpb;
      const int toks = (pr < 0) ? 0 : max(0, min(p.tpb, n_new - i0));
      int n = (toks > 0) ? nT : 0;
      if (p.causal && toks > 0) {
        const int seen = off + i0 + toks - 1;
        n = seen < 0 ? 0 : min(nT, seen / kTile + 1);
      }
      n = max(0, min(n, u.j1) - u.j0);
      u.n_pair = max(u.n_pair, n);
      if (t == static_cast<int>(rank)) {
        u.n_mine = n;
        u.toks = toks;
        u.tok = tok0 + i0;
        u.lim0 = p.causal ? off + i0 : kAllKeys;
      }
    }
    return u;
  };

  if (tid == 0) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&ctl->k_full[s], 1);
      mbar_init(&ctl->k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&ctl->v_full[s], 1);
      mbar_init(&ctl->v_empty[s], 1);
    }
    for (int s = 0; s < 6; ++s) {
      mbar_init(&ctl->s_full[s], 1);
      mbar_init(&ctl->s_free[s], 1);
    }
    for (int s = 0; s < kNB; ++s) {
      // this CTA's 4 warps + the score issuer's arrival (which sets the 16
      // bytes that CTA 1's 4 warps complete)
      mbar_init(&ctl->dec[s], kGroupWarps + 1);
    }
    for (int w = 0; w < kSoftWarps; ++w) {
      mbar_init(&ctl->drain[w], 1);
      mbar_init(&ctl->rescaled[0][w], 1);
      mbar_init(&ctl->rescaled[1][w], 1);
    }
    mbar_init(&ctl->o_full, 1);
    mbar_init(&ctl->o_free, kGroupWarps + 1);  // likewise, with 16 bytes from CTA 1
    mbar_init(&ctl->mma_done[0], 1);
    mbar_init(&ctl->mma_done[1], 1);
    mbar_init(&ctl->mma_done[2], 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ctl->handed[s], kGroupWarps);
      mbar_init(&ctl->summed[s], kGroupWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->q_full[s], 1);
      mbar_init(&ctl->q_empty[s], kTwo ? 2 : 1);
      mbar_init(&ctl->unit_full[s], 1);
      mbar_init(&ctl->unit_empty[s], kThreads / 32 - (leader ? 1 : kTwo ? 4 : 3));  // (CTA 1's issuers idle)
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->next_full[s], 1);
      mbar_init(&ctl->next_empty[s], 2);
    }
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc_pair(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish_pair();
  }
  if (p.B <= kSeqs)
    for (int i = tid; i <= p.B; i += kThreads) {
      ctl->cu[i] = __ldg(p.cu_seqlens + i);
      if (i < p.B) ctl->len[i] = __ldg(p.seq_lens + i);
    }
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait_pair(bar, parity, abort_flag, peer_abort);
  };
  // Waits of whole warps, and the next unit's geometry (i: units so far).
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };
  auto next_unit = [&](int i, Unit* u) -> bool {
    if (!wwait(&ctl->unit_full[i & 1], (i >> 1) & 1)) return false;
    *u = ctl->unit[i & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->unit_empty[i & 1]);
    return u->id >= 0;
  };
  // Outer coordinate in the pools of tiles jj + lane of a unit: page * Hkv +
  // KV head; a page outside the pool lies outside the map and reads zeros.
  auto pages32 = [&](const Unit& u, int jj) -> int {
    if (jj + lane >= u.n_pair) return 0;
    const int page = __ldg(p.page_table + static_cast<long>(u.b) * p.max_pages + u.j0 + jj + lane);
    return (page >= 0 && page < p.num_pages ? page : p.num_pages) * p.Hkv + u.kvh;
  };

  if (warp >= kSoftWarps) setmaxnreg_dec<kRegsDown<MODE>>();
  // The V tile jj of a unit (outer coordinate z) into its ring entry, by a whole warp.
  auto load_v = [&](const Unit& u, int jj, int z, uint32_t tc) -> bool {
    const uint32_t s = tc % NV;
    if (!wwait(&ctl->v_empty[s], ((tc / NV) & 1) ^ 1)) return false;
    if (lane == 0) {
      if (leader) mbar_arrive_expect_tx(&ctl->v_full[s], 2 * C::kVHalfBytes);
      tma_load_3d_pair(sV + s * C::kVHalfBytes, &tmV, lead(&ctl->v_full[s]), 64 * static_cast<int>(rank),
                       u.j0 + jj == u.last ? -u.last_shift : 0, z);
    }
    return true;
  };
  // Counters that every role keeps alike: tc, tiles before this unit; uc, units with tiles before it.
  if (warp == kWarpK) {
    // ------------------------------------------------------------ units, Q, K producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      if (kTwo) tma_prefetch_desc(&tmV);
    }
    int x = blockIdx.x >> 1;
    uint32_t tc = 0, uc = 0;
    for (int i = 0;; ++i) {
      // (the geometry's slot: read by all warps two units ago)
      if (!wwait(&ctl->unit_empty[i & 1], ((i >> 1) & 1) ^ 1)) break;
      Unit u;
      u.id = -1;
      if (x >= 0) u = geometry(x);
      if (lane == 0) {
        ctl->unit[i & 1] = u;
        mbar_arrive(&ctl->unit_full[i & 1]);
      }
      __syncwarp();
      if (x < 0) break;
      bool ok = true;
      int z = pages32(u, 0);
      if (u.n_pair > 0) {
        const uint32_t qs = uc & 1;
        ok = wwait(&ctl->q_empty[qs], ((uc >> 1) & 1) ^ 1);
        if (ok && lane == 0) {
          if (leader) mbar_arrive_expect_tx(&ctl->q_full[qs], 2 * C::kChunksQ * (p.tpb * p.G * 128));
          const uint32_t qbar = lead(&ctl->q_full[qs]);
#pragma unroll
          for (int c = 0; c < C::kChunksQ; ++c)
            tma_load_4d_pair(sQ + qs * C::kQBytes + c * (kTile * 128), &tmQ, qbar, c * 64, 0, u.kvh, u.tok);
        }
        ++uc;
      }
      // The next unit is asked for when the last tiles' loads of this one go
      // out, not before: a cluster that is far from done must not take what an
      // idle one could.  Both CTAs have read the answer before the last
      // (next_empty).
      const int ask_at = max(0, u.n_pair - NK);
      for (int jj = 0; ok && jj <= u.n_pair; ++jj) {
        if (jj == ask_at) {
          if (leader) ok = wwait(&ctl->next_empty[i & 1], ((i >> 1) & 1) ^ 1);
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&ctl->next_full[i & 1], 16);
            if (leader) request_cluster(ctl->answer[i & 1], &ctl->next_full[i & 1]);
          }
          __syncwarp();
        }
        if (jj == u.n_pair) break;
        if ((jj & 31) == 0 && jj > 0) z = pages32(u, jj);
        const int zt = __shfl_sync(0xffffffffu, z, jj & 31);
        const uint32_t s = tc % NK;
        if (ok) ok = wwait(&ctl->k_empty[s], ((tc / NK) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          if (leader) mbar_arrive_expect_tx(&ctl->k_full[s], 2 * C::kKHalfBytes);
          const uint32_t kbar = lead(&ctl->k_full[s]);
          const int y = 64 * static_cast<int>(rank) - (u.j0 + jj == u.last ? u.last_shift : 0);
#pragma unroll
          for (int c = 0; c < C::kChunksQ; ++c)
            tma_load_3d_pair(sK + s * C::kKHalfBytes + c * C::kKChunk, &tmK, kbar, c * 64, y, zt);
        }
        if constexpr (kTwo) {
          if (!(ok = load_v(u, jj, zt, tc))) break;
        }
        ++tc;
      }
      if (!ok) break;
      if (!wwait(&ctl->next_full[i & 1], (i >> 1) & 1)) break;
      x = requested_block(ctl->answer[i & 1]);
      x = x >= 0 ? x >> 1 : -1;
      __syncwarp();
      if (lane == 0) {  // read before the next answer lands
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (leader)
          mbar_arrive(&ctl->next_empty[i & 1]);
        else
          mbar_arrive_cluster(map_shared(smem_u32(&ctl->next_empty[i & 1]), 0u));
      }
    }
    __syncwarp();
  } else if (!kTwo && warp == kWarpV) {
    // ------------------------------------------------------------ V producer
    if (lane == 0) tma_prefetch_desc(&tmV);
    uint32_t tc = 0;
    Unit u;
    bool ok = true;
    for (int i = 0; ok && next_unit(i, &u); ++i) {
      int z = 0;
      for (int jj = 0; ok && jj < u.n_pair; ++jj, ++tc) {
        if ((jj & 31) == 0) z = pages32(u, jj);
        ok = load_v(u, jj, __shfl_sync(0xffffffffu, z, jj & 31), tc);
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma || warp == kWarpV) {
    // ------------------------------------------------------------ score issuer(s) (leader)
    // Between a tile's MMAs and the next one's, the issuer commits and waits
    // for some 300 cycles.  In the dense path P.V fills them; with the vote,
    // where most tiles have no P.V, two issuers take alternate tiles (0: the
    // even ones), so that one's MMAs run while the other synchronises.
    const uint32_t me = (kTwo && warp == kWarpV) ? 1 : 0;
    constexpr uint32_t kStep = kTwo ? 2 : 1;
    constexpr uint32_t idS = idesc_bf16_f32(256, 128, false, false);
    const uint64_t dq = smem_desc(smem_u32(sQ), 16, 1024);
    const uint32_t sKa = smem_u32(sK);
    uint32_t tc = 0, uc = 0;
    Ring<NK, kStep> rk{me};
    Ring<kSlots, kStep> rt{me}, rf{(me + kNB) % kSlots, 1};  // slots of the tile; of the one three before it
    uint32_t col = 128u * me;  // its score buffer
    Unit u;
    bool ok = true;
    for (int i = 0; leader && ok && next_unit(i, &u); ++i) {
      if (u.n_pair == 0) continue;
      if (lane == 0) {
        ok = wait(&ctl->q_full[uc & 1], (uc >> 1) & 1);
        const uint64_t dqu = dq + (((uc & 1) * C::kQBytes) >> 4);
        for (uint32_t t = tc + (kTwo ? (me ^ (tc & 1)) : 0); ok && t < tc + u.n_pair; t += kStep) {
          if (!(ok = wait(&ctl->k_full[rk.at], rk.par))) break;
          // The buffer's previous tile, three before, has been decided by both
          // blocks and its P.V (if any) issued: S_t is ordered after it
          // (tcgen05 fence + barrier).
          if (!(ok = wait(&ctl->s_free[rf.at], rf.par))) break;
          tc_fence_after();
          const uint64_t dk = smem_desc(sKa + rk.at * C::kKHalfBytes, 16, 1024);
          if (!kTwo) col = 128u * rt.at;
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk) {
            const uint32_t qoff = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
            const uint32_t koff = ((kk >> 2) * C::kKChunk + (kk & 3) * 32) >> 4;
            mma2_bf16_ss(tmem + col, dqu + qoff, dk + koff, idS, kk > 0 ? 1u : 0u);
          }
          mma2_commit_mc(&ctl->s_full[rt.at], 3);
          mma2_commit_mc(&ctl->k_empty[rk.at], 3);
          // CTA 1's four warps on this tile complete 4 bytes each on dec; this
          // arrival sets that count for the tile's phase.
          mbar_arrive_expect_tx(&ctl->dec[kTwo ? col >> 7 : rt.at], 4 * kGroupWarps);
          rk.next();
          rt.next();
          rf.next();
          if (kTwo && (col += 256u) >= 384u) col -= 384u;
        }
        if (ok) mma2_commit_mc(&ctl->q_empty[uc & 1], 3);
      }
      tc += u.n_pair;
      ++uc;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (leader && lane == 0) {
      // Every MMA issued must have finished before TMEM is freed.
      const int d = me ? 2 : 0;
      mma2_commit_mc(&ctl->mma_done[d], 1);
      mbar_wait(&ctl->mma_done[d], 0, nullptr);
    }
    __syncwarp();
  } else if (warp == kWarpPV) {
    // ------------------------------------------------------------ P.V issuer (leader)
    constexpr uint32_t idO = idesc_bf16_f32(256, DV, false, true);
    const uint32_t sVa = smem_u32(sV);
    uint32_t tc = 0, uc = 0;
    uint32_t nresc = 0u;  // bit (kSoftWarps * r + warp): parity of (CTA r, warp)'s requests
    Unit u;
    bool ok = true;
    for (int i = 0; leader && ok && next_unit(i, &u); ++i) {
      if (u.n_pair == 0) continue;
      if (lane == 0) {
        // O is read by the last unit's epilogue (of CTA 1's warps: as bytes).
        if (uc > 0) ok = wait(&ctl->o_free, (uc - 1) & 1);
        mbar_arrive_expect_tx(&ctl->o_free, 4 * kGroupWarps);
        uint32_t o_acc = 0u;
        for (int jj = 0; ok && jj < u.n_pair; ++jj, ++tc) {
          const uint32_t bsel = tc % kNB;
          const uint32_t ph = (tc / kNB) & 1;
          // The tile's V halves do not depend on the decisions: wait for them
          // first, while the softmax is still deciding.
          const uint32_t vs = tc % NV;
          if (!(ok = wait(&ctl->v_full[vs], (tc / NV) & 1))) break;
          if (!(ok = wait(&ctl->dec[bsel], ph))) break;
          // (plain loads: the barrier waits above are compiler memory barriers)
          const uint4 f4 = *reinterpret_cast<const uint4*>(ctl->flags[bsel]);
          const uint4 g4 = *reinterpret_cast<const uint4*>(ctl->peer_flags[bsel]);
          const uint32_t any = f4.x | f4.y | f4.z | f4.w | g4.x | g4.y | g4.z | g4.w;
          if (any & kFlagRescale) {
            // The tile's decisions come from the warps of warpgroup tc % 2.
            const int wg0 = kGroupWarps * (tc & 1);
            const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
            const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w};
            uint32_t resc = 0u;  // bit (kGroupWarps * r + w)
#pragma unroll
            for (int w = 0; w < kGroupWarps; ++w) {
              resc |= ((f[w] >> 1) & 1u) << w;
              resc |= ((g[w] >> 1) & 1u) << (kGroupWarps + w);
            }
            // Warps that move their reference maximum rescale O once every P.V
            // issued so far has finished.
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int w = 0; w < kGroupWarps; ++w)
                if (resc & (1u << (kGroupWarps * r + w)))
                  mma2_commit_mc(&ctl->drain[wg0 + w], static_cast<uint16_t>(1u << r));
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int w = 0; w < kGroupWarps; ++w) {
                const uint32_t bit = 1u << (kSoftWarps * r + wg0 + w);
                if (ok && (resc & (1u << (kGroupWarps * r + w)))) {
                  const uint32_t par = (nresc & bit) ? 1u : 0u;
                  ok = (r == 0) ? wait(&ctl->rescaled[0][wg0 + w], par)
                                : mbar_wait_pair<true>(&ctl->rescaled[1][wg0 + w], par, abort_flag,
                                                       peer_abort);
                  nresc ^= bit;
                }
              }
            if (!ok) break;
          }
          // (The first tile's P.V sets O, of zeros if no block kept it: NaN queries.)
          if ((any & kFlagKept) || o_acc == 0u) {
            tc_fence_after();
            const uint64_t dv = smem_desc(sVa + vs * C::kVHalfBytes, 16384, 1024);
            const uint32_t pcol = 128u * bsel;
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)  // P of keys 16kk..: column 64 (kk / 4) + 8 (kk % 4)
              mma2_bf16_ts(tmem + C::kColO, tmem + pcol + 64 * (kk >> 2) + 8 * (kk & 3),
                           dv + ((kk * 2048) >> 4), idO, (o_acc | kk) ? 1u : 0u);
            o_acc = 1u;
          }
          tc_fence_before();
          mbar_arrive(&ctl->s_free[tc % kSlots]);
          mma2_commit_mc(&ctl->v_empty[vs], 3);
        }
        if (ok) mma2_commit_mc(&ctl->o_full, 3);
      }
      ++uc;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (leader && lane == 0) {
      mma2_commit_mc(&ctl->mma_done[1], 1);
      mbar_wait(&ctl->mma_done[1], 0, nullptr);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax / vote
    // Two warpgroups take alternate tiles: warpgroup g = warp / 4 those with an
    // even / odd number over all units, one thread per row (warp w reads TMEM
    // lanes 32 (w % 4) .. + 31) over all 128 score columns, loaded as two
    // halves of 64.  Within a unit a row's running state passes from one
    // warpgroup to the other once per tile: the warpgroup on a tile writes the
    // running maximum m of the vote and the reference maximum m_ref of P to
    // shared memory and its warps arrive on a barrier, which the other
    // completes before its next vote.  Each warpgroup sums its own tiles' P
    // into l against the m_ref it last saw; a moved m_ref rescales that sum
    // when the state arrives.  The warpgroup with the unit's last tile adds the
    // other's sum (`fin`) and writes the output, while the other is already at
    // the next unit's first tile.  How far one may run ahead of the other is
    // bounded by the three score buffers and the one O: tile t + 4 needs the
    // buffer of t + 1, whose P.V waits for the O of t's unit to be read.  So
    // four slots of each shared array are enough.
    // Threads leave together per warpgroup (agreed on at the start of a unit);
    // all waits on the other warpgroup are bounded.
    setmaxnreg_inc<kRegsUp<MODE>>();
    const int g = warp / kGroupWarps, q4 = warp % kGroupWarps;
    const int row = q4 * 32 + lane;  // TMEM lane
    const int gtid = tid - 128 * g;  // thread index within the warpgroup
    const int tok = row / p.G, head = row - tok * p.G;  // of the block, of the group
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    const uint32_t colO = lane_base + C::kColO;
    const float sl2 = p.scale_log2;
    uint32_t n_drain = 0;
    const uint32_t bar_vote = 5 + g;           // the 128 threads of this warpgroup
    uint32_t tc = 0, uc = 0;
    Unit u;
    bool ok = true;
    for (int i = 0;; ++i) {
      const bool have = next_unit(i, &u);
      if (named_bar_or(bar_vote, 128, !(ok && have))) break;
      const bool row_valid = tok < u.toks;
      // Last key index this row may see.  A row without a token is not masked:
      // it takes no part in the vote, and nothing of it is kept.
      const int lim = row_valid ? min(u.last * kTile + kTile - 1 - u.last_shift, u.lim0 + tok) : kAllKeys;
      const long unit_row = static_cast<long>(u.id) * p.max_pages;
      float m_true = -INFINITY, m_ref = -INFINITY, l = 0.f;
      uint32_t skipped = 0;
      const int jj0 = (g ^ tc) & 1;                                 // this warpgroup's first tile
      const bool owner = ((tc + max(u.n_pair, 1) - 1) & 1) == g;    // it has the last one
      int in_range = jj0;  // tile jj's place in its range of the vote
      if (kVote)
        while (in_range >= u.range) in_range -= u.range;

      // Columns 64 hf .. + 63 of the scores of tile j, masked, into sr; returns their maximum.
      auto load_half = [&](uint32_t colS, int j, int hf, uint32_t* sr) -> float {
        tmem_ld32p(colS + 64 * hf, sr);
        tmem_ld32p(colS + 64 * hf + 32, sr + 32);
        tmem_wait_ld();
        // Column e of the half is key k0 + e; the last tile's first columns are no keys.
        const int shift = (j == u.last) ? u.last_shift : 0;
        const int first = shift - 64 * hf, vis = lim - (j * kTile - first);
        if (first > 0 || vis < 63) {
          // bit e: column e is seen (a bit test a column; two comparisons: 406 us
          // for the mixed step of 48 sequences, so 399)
          const uint64_t upto = vis >= 63 ? ~0ull : vis < 0 ? 0ull : (2ull << vis) - 1;
          const uint64_t seen = upto & (first >= 64 ? 0ull : first > 0 ? ~0ull << first : ~0ull);
          const uint32_t lo = static_cast<uint32_t>(seen), hi = static_cast<uint32_t>(seen >> 32);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (!(lo & (1u << e))) sr[e] = __float_as_uint(-INFINITY);
            if (!(hi & (1u << e))) sr[32 + e] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          mx[e & 3] = fmax3(mx[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      };
      // P = exp2(s*scale*log2e - m_ref*scale*log2e) of the 64 scores in sr, as
      // bf16 pairs into sr[0..31]; returns their sum.
      auto exp_half = [&](uint32_t* sr) -> float {
        const float mb = (m_ref == -INFINITY) ? 0.f : m_ref * sl2;
        const uint64_t sl2x2 = f32x2(sl2, sl2), nmb = f32x2(-mb, -mb);
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int cc = 8 * q; cc < 8 * q + 8; ++cc) {
            const uint64_t xp = fma_f32x2(
                f32x2(__uint_as_float(sr[2 * cc]), __uint_as_float(sr[2 * cc + 1])), sl2x2, nmb);
            const float p0 = ex2_approx(f32x2_lo(xp));
            const float p1 = ex2_approx(f32x2_hi(xp));
            ls[cc & 1] = add_f32x2(ls[cc & 1], f32x2(p0, p1));
            sr[cc] = pack_bf16x2(p0, p1);
          }
          if (q < 3) order_after(sr + 8 * q, sr + 16 * (q + 1));
        }
        const uint64_t lsum = add_f32x2(ls[0], ls[1]);
        return f32x2_lo(lsum) + f32x2_hi(lsum);
      };

      for (int jj = jj0; jj < u.n_pair; jj += 2) {
        const int j = u.j0 + jj;  // tile of the sequence
        const uint32_t t = tc + jj, bsel = t % kNB;
        const uint32_t colS = lane_base + 128u * bsel;
        if (!wwait(&ctl->s_full[t % kSlots], (t / kSlots) & 1)) ok = false;
        tc_fence_after();
        const bool mine = jj < u.n_mine;
        uint32_t sr[64];
        float tmax = -INFINITY;
        if (mine) {
          const bool masked = j == u.last || lim < j * kTile + kTile - 1;
          if ((kVote || DQK == 64) && !__any_sync(0xffffffffu, masked)) {
            // No lane of the warp masks a column: all 128 at once.  With the vote most
            // tiles end here, at d = 64 the matrix work is short: one wait for the
            // loads instead of two (4 x 2K on 32K with the skip test 1.98 -> 1.95 ms,
            // mixed step 414 -> 406 us, cross attention 45 -> 43 us).  The dense path
            // at d = 128 is bound elsewhere and loses 4% to the larger code.
            uint32_t s0[64];
            tmem_ld32p(colS, s0);
            tmem_ld32p(colS + 32, s0 + 32);
            tmem_ld32p(colS + 64, sr);
            tmem_ld32p(colS + 96, sr + 32);
            tmem_wait_ld();
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              mx[e & 3] = fmax3(mx[e & 3], __uint_as_float(s0[2 * e]), __uint_as_float(s0[2 * e + 1]));
              mx[(e + 2) & 3] = fmax3(mx[(e + 2) & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
            }
            tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          } else {
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) tmax = fmaxf(tmax, load_half(colS, j, hf, sr));  // sr keeps the second half
          }
          if (!row_valid) tmax = -INFINITY;
        }
        // The state after the previous tile, from the other warpgroup.
        if (jj > 0) {
          if (!wwait(&ctl->handed[(t - 1) & 3], ((t - 1) >> 2) & 1)) ok = false;
          const float2 hs = ctl->hand[(t - 1) & 3][row];
          m_true = hs.x;
          if (hs.y != m_ref) {
            if (m_ref != -INFINITY) l *= ex2_approx((m_ref - hs.y) * sl2);
            m_ref = hs.y;
          }
        }
        bool kept = false, resc = false, first = false;
        float alpha = 1.f;
        if constexpr (kVote) {
          // A range of the vote starts without a running maximum.
          first = in_range == 0;
          if (first) m_true = -INFINITY;
          in_range += 2;
          while (in_range >= u.range) in_range -= u.range;
        }
        if (mine) {
          // Skip vote: every row of the block must pass exp(scale*(tile_max - m)) < lambda.
          // No row passes at a range's first tile.  (Some row sees a key there; but if the rows
          // are all NaN, which the maximum drops, no other tile is kept, and they stay NaN.)
          float c = first ? INFINITY : -INFINITY;
          if (tmax != -INFINITY) c = (m_true == -INFINITY) ? INFINITY : tmax - m_true;
          if constexpr (kVote) {
            kept = !named_bar_and(bar_vote, 128, c < u.thr_raw);
            if (p.margin != nullptr) {
              float cm = c;
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, o));
              if (lane == 0) *reinterpret_cast<volatile float*>(&ctl->red[g][q4]) = cm;
              named_bar_sync(bar_vote, 128);
              if (gtid == 0) {
                const volatile float* rr = ctl->red[g];
                const float cmax = fmaxf(fmaxf(rr[0], rr[1]), fmaxf(rr[2], rr[3]));
                p.margin[unit_row + j] = (cmax == INFINITY) ? INFINITY : cmax * p.scale;
              }
            }
            if (gtid == 0) {
              skipped += kept ? 0u : 1u;
              if (p.mask != nullptr) p.mask[unit_row + j] = kept ? 0 : 1;
            }
          } else {
            kept = true;
          }
          m_true = fmaxf(m_true, tmax);
          if (kept) {
            // m_ref trails m lazily: it moves only when m has grown by more than
            // 2^8 in exp2 units, and then the warp's rows of O are rescaled.
            bool need = false;
            if (m_ref == -INFINITY) {
              m_ref = m_true;  // no key of this row counted yet: its O row and l are zero
            } else if ((m_true - m_ref) * sl2 > kRescaleLog2) {
              need = true;
            }
            resc = __any_sync(0xffffffffu, need);
            if (resc && m_ref != -INFINITY && m_true > m_ref) {
              alpha = ex2_approx((m_ref - m_true) * sl2);
              l *= alpha;
              m_ref = m_true;
            }
          }
        }
        ctl->hand[t & 3][row] = make_float2(m_true, m_ref);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->handed[t & 3]);
        // P of columns 64 hf .. as bf16 pairs over the first 32 of those score
        // columns; the second half goes first, from the registers, then the
        // first half is loaded again.  A skipped or unseen tile writes zeros
        // (the pair's P.V covers both blocks; the other block may keep the tile).
        if (kept) {
#pragma unroll(DQK == 64 ? 1 : 2)
          for (int hf = 1; hf >= 0; --hf) {
            if (hf == 0) load_half(colS, j, 0, sr);
            l += exp_half(sr);
            tmem_st32p(colS + 64 * hf, sr);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) sr[e] = 0u;
          tmem_st32p(colS + 64, sr);
          tmem_st32p(colS, sr);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t f = (kept ? kFlagKept : 0u) | (resc ? kFlagRescale : 0u);
          if (leader) {
            *reinterpret_cast<volatile uint32_t*>(&ctl->flags[bsel][q4]) = f;
            mbar_arrive(&ctl->dec[bsel]);
          } else {
            st_async_u32(map_shared(smem_u32(&ctl->peer_flags[bsel][q4]), 0u), f,
                         lead(&ctl->dec[bsel]));
          }
        }
        if (resc) {
          // The P.V issuer drains the P.V MMAs issued so far; then this warp's
          // rows of O are rescaled before this tile's P.V.
          if (!wwait(&ctl->drain[warp], n_drain & 1)) ok = false;
          ++n_drain;
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < DV / 32; ++cc) {
              uint32_t orr[32];
              tmem_ld32p(colO + cc * 32, orr);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
              tmem_st32p(colO + cc * 32, orr);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (leader)
              mbar_arrive(&ctl->rescaled[0][warp]);
            else
              mbar_arrive_cluster(lead(&ctl->rescaled[1][warp]));
          }
        }
      }
      tc += u.n_pair;

      const uint32_t fs = uc & 3;
      if (!owner) {
        if (u.n_pair > 0) {
          ctl->fin[fs][row] = make_float2(m_ref, l);
          if (gtid == 0) ctl->skipped[fs] = skipped;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->summed[fs]);
          ++uc;
        }
        continue;
      }
      // The row's denominator: both warpgroups' sums against m_ref, the one O
      // is kept against (this warpgroup has it from the last tile).
      float l_row = l;
      if (u.n_pair > 0) {
        if (!wwait(&ctl->summed[fs], (uc >> 2) & 1)) ok = false;
        const float2 other = ctl->fin[fs][row];
        // (A sum of zero may stand against no maximum; that of a NaN row is NaN.)
        if (other.y != 0.f) l_row += other.y * ex2_approx((other.x - m_ref) * sl2);
        if (!wwait(&ctl->o_full, uc & 1)) ok = false;
        ++uc;
        tc_fence_after();
      }

      // Epilogue: the rows' O as O / l in bf16 (a row that saw no key writes
      // zeros), or of a part as it is, in fp32.
      const bool writes = ok && row_valid;
      const size_t orow = static_cast<size_t>(u.tok + tok) * p.Hq + u.kvh * p.G + head;
      const size_t rows = static_cast<size_t>(p.T) * p.Hq;
      if (writes && p.parts > 1) p.part_ml[u.part * rows + orow] = make_float2(m_ref * sl2, l_row);
      const float inv_l = (l_row != 0.f) ? 1.f / l_row : 0.f;  // (NaN stays NaN)
#pragma unroll
      for (int c = 0; c < DVO / 64; ++c) {
        uint32_t orr[64];
        if (u.n_pair > 0) {
          tmem_ld32p(colO + c * 64, orr);
          tmem_ld32p(colO + c * 64 + 32, orr + 32);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) orr[e] = 0u;
        }
        if (u.n_pair > 0 && c == DVO / 64 - 1) {  // O may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (leader)
              mbar_arrive(&ctl->o_free);
            else
              st_async_u32(map_shared(smem_u32(&ctl->o_note[q4]), 0u), 0u, lead(&ctl->o_free));
          }
        }
        if (writes) {
          if (p.parts > 1) {
            if (l_row != 0.f) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + (u.part * rows + orow) * DVO + c * 64);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                dst[e] = make_float4(__uint_as_float(orr[4 * e]), __uint_as_float(orr[4 * e + 1]),
                                     __uint_as_float(orr[4 * e + 2]), __uint_as_float(orr[4 * e + 3]));
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.o + orow * DVO + c * 64);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                v[k] = pack_bf16x2(__uint_as_float(orr[8 * e + 2 * k]) * inv_l,
                                   __uint_as_float(orr[8 * e + 2 * k + 1]) * inv_l);
              dst[e] = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
      }
      // Debug outputs: the unit's count, and the tiles that it does not see.
      if (kVote && gtid == 0 && p.counts != nullptr) {
        const uint32_t n = skipped + (u.n_pair > 0 ? ctl->skipped[fs] : 0u);
        if (p.parts == 1)
          p.counts[u.id] = n;
        else
          atomicAdd(p.counts + u.id, n);  // (cleared before the launch)
      }
      if (p.mask != nullptr || p.margin != nullptr) {
        const int end = u.part == p.parts - 1 ? p.max_pages : u.j1;
        for (int j = u.j0 + u.n_mine + gtid; j < end; j += 128) {
          if (p.mask != nullptr) p.mask[unit_row + j] = 2;
          if (p.margin != nullptr) p.margin[unit_row + j] = NAN;
        }
      }
      __syncwarp();
    }
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  // After an expired wait, copies may still be in flight into either CTA's
  // shared memory (the leader's barriers count both halves; a requested unit's
  // number): give them time to land before the pair's shared memory is released.
  if (*abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000ull) {
    }
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
  if (tid == 0 && *abort_flag) report_timeout(p.status);
}

// Joins a row's partial states: o = sum_s 2^(m_s - m*) O_s / sum_s 2^(m_s -
// m*) l_s, m* the largest m of the parts that kept a key.  A warp per row; rows
// of tokens that belong to no sequence are left as they were.
template <int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p) {
  const long rows = static_cast<long>(p.T) * p.Hq;
  const long row = static_cast<long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int tok = static_cast<int>(row / p.Hq);
  if (tok >= p.T || tok < p.cu_seqlens[0] || tok >= p.cu_seqlens[p.B]) return;
  float mstar = -INFINITY;
  for (int s = 0; s < p.parts; ++s) {
    const float2 ml = p.part_ml[s * rows + row];
    if (ml.y != 0.f) mstar = fmaxf(mstar, ml.x);
  }
  constexpr int E = D / 32;  // a lane's columns: E lane .. + E - 1
  float acc[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int s = 0; s < p.parts; ++s) {
    const float2 ml = p.part_ml[s * rows + row];
    if (ml.y == 0.f) continue;
    const float w = ex2_approx(ml.x - mstar);
    l = fmaf(ml.y, w, l);
    const float* src = p.part_o + (s * rows + row) * D + E * lane;
    float v[E];
    if constexpr (E == 4) {
      const float4 f = *reinterpret_cast<const float4*>(src);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(src);
      v[0] = f.x, v[1] = f.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(v[e], w, acc[e]);
  }
  const float inv = (l != 0.f) ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + E * lane);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
}

template <int D, Mode MODE>
cudaError_t launch_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const ChunkParams& p, cudaStream_t st) {
  using C = PairCfg<D, 128>;
  auto* fn = chunk_paged_kernel<D, 128, D, MODE>;
  // With fewer registers at launch the softmax warpgroups' increase could
  // never be satisfied: refuse to launch in that case.
  static const int launch_regs = [fn] {
    cudaFuncAttributes attr{};
    return cudaFuncGetAttributes(&attr, fn) == cudaSuccess ? attr.numRegs : -1;
  }();
  if (launch_regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  // One cluster per unit; those that are not launched yet are taken over by running ones.
  const long units = static_cast<long>(p.slots) * p.Hkv * p.parts;
  if (p.counts != nullptr && (p.parts > 1 || MODE == Mode::kDense)) {
    e = cudaMemsetAsync(p.counts, 0, sizeof(uint32_t) * 2 * p.slots * p.Hkv, st);
    if (e != cudaSuccess) return e;
  }
  fn<<<dim3(static_cast<unsigned>(2 * units)), dim3(kThreads), C::kSmemBytes, st>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.parts == 1) return e;
  const long rows = static_cast<long>(p.T) * p.Hq;
  chunk_merge_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Parts of the tiles.  A part's states are written and merged again (a second
// kernel, ~6 us in all), so parts are made only where the pairs leave places
// of the 76 clusters idle, at most as many as fit at once, and of eight tiles
// or more.  Measured on 8 sequences x 5 new tokens x 2K keys (64 pairs, 8 KV
// heads): 24 us as one part, 29 us as two.
int chunk_parts(long pairs, int S, int max_pages) {
  const long places = 76;
  long parts = places / pairs;
  if (parts > max_pages / 8) parts = max_pages / 8;
  return parts < 1 ? 1 : parts < S ? static_cast<int>(parts) : S;
}

cudaError_t launch_chunk_paged(int d, bool vote, const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, const ChunkParams& p, cudaStream_t st) {
  if (d == 128)
    return vote ? launch_chunk<128, Mode::kSparse>(tq, tk, tv, p, st)
                : launch_chunk<128, Mode::kDense>(tq, tk, tv, p, st);
  return vote ? launch_chunk<64, Mode::kSparse>(tq, tk, tv, p, st)
              : launch_chunk<64, Mode::kDense>(tq, tk, tv, p, st);
}

}  // namespace ssattn

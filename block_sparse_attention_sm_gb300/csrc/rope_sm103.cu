// Rotary positions of query and key rows, alone or fused with the write of a
// step's new keys and values into the paged cache.
//
// A row's entries [off, off + rot) are rot / 2 pairs (a, b); at position p the
// pair i turns by the angle p * w_i:
//   a' = f (a cos - b sin),  b' = f (b cos + a sin)
// (f: a factor on cosines and sines; the transposed rotation, which is the
// gradient, has the sines negated).  Pairs are (i, i + rot / 2) or adjacent.
//
// The angle is formed exactly: w / 2 pi, the turns per position, as a 64-bit
// binary fraction, so that p times it modulo 2^64 is the fractional turn of
// any 32-bit position with an error below 2^-32 turns for |w| < 2 (the usual
// frequencies are at most 1; each doubling beyond doubles the error; from 2^64
// on no bit of the angle is left at any position, and the result is NaN, as it
// is where w is not finite).  (fp32 products lose the
// angle of far positions: 2^-24 of 10^5 radians is 6e-3.)  Integer products
// only: fp64 runs at 1/64 of the fp32 rate on this GPU.  The fraction's upper
// 32 bits become a float in half turns for sincospif; its rounding (2^-25
// turns' relative) and bf16's of the result (half a step, 2^-8) are the only
// ones.
//
// Bound by memory: 4 bytes per entry, read and written once.  A block takes
// TB tokens; a thread one column of a token (8 pairs, or 4 adjacent ones:
// 16-byte accesses) for every HS-th head, with the first heads' loads in
// flight while the block forms the tokens' angles, each once, in shared
// memory (a sincospif costs as much as moving a few heads' entries).
#include "rope.cuh"

#include "common.cuh"

namespace ssattn {
namespace {

constexpr int kThreadsRope = 256;
constexpr int kAhead = 4;  // heads whose loads are in flight per thread

// Binary exponent: 2^e <= |w| < 2^(e + 1); above every finite one for NaN and Inf.
__device__ __forceinline__ int exponent_of(double w) {
  return static_cast<int>((static_cast<uint64_t>(__double_as_longlong(w)) >> 52) & 0x7ff) - 1023;
}

// w / (2 pi) modulo 1 as a fraction of 2^64 (truncated).
__device__ __forceinline__ uint64_t turns_per_position(double w) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(w));
  const int e = exponent_of(w);
  const uint64_t m = (bits << 11) | (1ull << 63);           // |w| = m 2^(e - 63)
  const uint64_t inv2pi = 0xA2F9836E4E441529ull;            // 2^66 / (2 pi), truncated
  const uint64_t t = __umul64hi(m, inv2pi);                 // |w| / 2 pi = t 2^(e - 65)
  uint64_t f = 0;
  if (e >= 1)
    f = (e - 1 < 64) ? t << (e - 1) : 0;
  else if (1 - e < 64)
    f = t >> (1 - e);
  return (bits >> 63) ? 0ull - f : f;
}

// Cosine and sine (times the factor) of position `pos` at frequency `w`.
__device__ __forceinline__ float2 turn_of(int pos, double w, float factor, float sign) {
  const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns_per_position(w);
  const float half_turns = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 4.656612873077393e-10f;
  float s, c;
  sincospif(half_turns, &s, &c);
  if (exponent_of(w) >= 64) factor = NAN;  // (a select; a branch around the angle: decode append +0.2 us)
  return make_float2(factor * c, sign * factor * s);
}

// The products are contracted the same way in every form of the kernel, so
// that alignment and layout do not change a bit of the results.
__device__ __forceinline__ float turned_a(float a, float b, float2 cs) {
  return fmaf(a, cs.x, -__fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turned_b(float a, float b, float2 cs) {
  return fmaf(b, cs.x, __fmul_rn(a, cs.y));
}

template <int N>
struct Chunk;  // N bf16 values in one access
template <>
struct Chunk<8> {
  uint4 v;
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
  __device__ __forceinline__ static Chunk load(const __nv_bfloat16* p) {
    return {*reinterpret_cast<const uint4*>(p)};
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Chunk<1> {
  __nv_bfloat16 v;
  __device__ __forceinline__ void get(float* f) const { f[0] = __bfloat162float(v); }
  __device__ __forceinline__ void set(const float* f) { v = __float2bfloat16_rn(f[0]); }
  __device__ __forceinline__ static Chunk load(const __nv_bfloat16* p) { return {*p}; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = v; }
};

// One column of a row: the pairs a thread turns, or entries it copies.
// VEC: 8-entry (16-byte) accesses; otherwise single entries.
// Split pairs: chunk a at `at`, chunk b at `at + rot / 2`.  Adjacent pairs:
// VEC holds 4 pairs in chunk a (chunk b unused); the single-entry form holds
// one pair as chunks a and b, one entry apart.
template <bool VEC, bool ADJ>
struct Column {
  static constexpr int kN = VEC ? 8 : 1;             // entries per chunk
  static constexpr int kPairs = VEC ? (ADJ ? 4 : 8) : 1;
  static constexpr bool kTwo = !(VEC && ADJ);        // uses chunk b
  using Ch = Chunk<kN>;
  int at, second;  // entry of chunk a; distance of chunk b
  bool turns;
  float2 cs[kPairs];

  // Columns of a row: rot / 2 / kPairs that turn, then the copied ones (none in place).
  __host__ __device__ static int turning(int rot) { return rot / 2 / kPairs; }
  __device__ __forceinline__ void place(int col, const RopeTurn& t) {
    const int n = turning(t.rot);
    turns = col < n;
    if (turns) {
      at = t.off + (ADJ ? (VEC ? 8 : 2) * col : kN * col);
      second = ADJ ? 1 : t.rot / 2;
    } else {
      at = kN * (col - n);
      if (at >= t.off) at += t.rot;
      second = 0;
    }
  }
  // This column's angles, from the block's table: entry i of column c of a
  // token at [(token * kPairs + i) * width + c].
  __device__ __forceinline__ void angles(const float2* table, int token, int c, int width) {
    if (turns) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) cs[i] = table[(token * kPairs + i) * width + c];
    }
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* row, Ch& a, Ch& b) const {
    a = Ch::load(row + at);
    if (kTwo && turns) b = Ch::load(row + at + second);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, const Ch& a, const Ch& b) const {
    a.store(row + at);
    if (kTwo && turns) b.store(row + at + second);
  }
  __device__ __forceinline__ void turn(Ch& a, Ch& b) const {
    if (!turns) return;
    float fa[kN], fb[kN];
    a.get(fa);
    if constexpr (kTwo) {
      b.get(fb);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float u = fa[i], w = fb[i];
        fa[i] = turned_a(u, w, cs[i]);
        fb[i] = turned_b(u, w, cs[i]);
      }
      b.set(fb);
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float u = fa[2 * i], w = fa[2 * i + 1];
        fa[2 * i] = turned_a(u, w, cs[i]);
        fa[2 * i + 1] = turned_b(u, w, cs[i]);
      }
    }
    a.set(fa);
  }
};

// Forms the block's table: the angles of `width` columns from `col0` on, of
// `tokens` tokens at the positions pos[].
template <class C>
__device__ __forceinline__ void fill_table(float2* table, const RopeTurn& t, const int* pos, int tokens,
                                           int col0, int width) {
  const int turning = min(width, max(0, C::turning(t.rot) - col0)) * C::kPairs;  // of each token
  for (int e = threadIdx.x; e < tokens * turning; e += kThreadsRope) {
    const int token = e / turning, pair = e - token * turning;
    const int c = pair / C::kPairs, i = pair - c * C::kPairs;
    table[(token * C::kPairs + i) * width + c] =
        turn_of(pos[token], __ldg(t.inv_freq + col0 * C::kPairs + pair), t.factor, t.sign);
  }
}

// A block: TB tokens x HS threads a column x `width` columns (of `cols`;
// blockIdx.y steps over wider rows).
template <bool VEC, bool ADJ>
__global__ void __launch_bounds__(kThreadsRope)
    rope_kernel(const RopeParams p, int cols, int width, int HS, int TB) {
  using C = Column<VEC, ADJ>;
  __shared__ float2 table[kThreadsRope * C::kPairs];
  __shared__ int pos[kThreadsRope];
  const int tid = threadIdx.x, per_token = width * HS;
  const long tokens = static_cast<long>(p.B) * p.L, t0 = static_cast<long>(blockIdx.x) * TB;
  const int here = static_cast<int>(min(static_cast<long>(TB), tokens - t0));
  const int ti = tid / per_token, rest = tid - ti * per_token;
  const int h0 = rest / width, cw = rest - h0 * width, col = cw + blockIdx.y * width;
  const bool mine = ti < here && col < cols;
  const long token = t0 + ti, b = token / p.L, l = token - b * p.L;
  const __nv_bfloat16* x = p.x + b * p.xs[0] + l * p.xs[2];
  __nv_bfloat16* out = p.out + b * p.os[0] + l * p.os[2];
  C c;
  c.place(col, p.turn);
  typename C::Ch a[kAhead], bb[kAhead];
  if (mine) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (h0 + u * HS < p.H) c.load(x + (h0 + u * HS) * p.xs[1], a[u], bb[u]);
  }
  if (tid < here) {
    const long tt = t0 + tid, tb = tt / p.L;
    pos[tid] = p.pos[tb * p.pos_stride + (tt - tb * p.L)];
  }
  __syncthreads();
  fill_table<C>(table, p.turn, pos, here, blockIdx.y * width, width);
  __syncthreads();
  if (!mine) return;
  c.angles(table, ti, cw, width);
  for (int h = h0;;) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (h + u * HS < p.H) {
        c.turn(a[u], bb[u]);
        c.store(out + (h + u * HS) * p.os[1], a[u], bb[u]);
      }
    h += kAhead * HS;
    if (h >= p.H) break;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (h + u * HS < p.H) c.load(x + (h + u * HS) * p.xs[1], a[u], bb[u]);
  }
}

// Rotation and cache write of a step's new tokens.  Token t of the packed
// batch belongs to the sequence b with cu[b] <= t < cu[b + 1]; it is the
// sequence's key number L_b - (cu[b + 1] - t).  "Heads" of a token here: its
// query heads, then its key heads (both turned), then its value heads
// (copied).  Tokens of no sequence (t >= cu[B]) are left alone, and a key
// whose page is missing is not written.
template <bool VEC, bool ADJ>
__global__ void __launch_bounds__(kThreadsRope)
    rope_append_kernel(const AppendParams p, int cols, int width, int HS, int TB) {
  using C = Column<VEC, ADJ>;
  __shared__ float2 table[kThreadsRope * C::kPairs];
  __shared__ int marks[kThreadsRope], pos[kThreadsRope], page[kThreadsRope], row[kThreadsRope];
  const int tid = threadIdx.x;
  const int per_token = width * HS;
  const int t0 = blockIdx.x * TB;  // this block's tokens
  const int ti = tid / per_token;  // (threads beyond TB tokens only help to count)
  const int t = t0 + ti;
  const int rest = tid - ti * per_token;
  const int h0 = rest / width, cw = rest - h0 * width, col = cw + blockIdx.y * width;
  const bool mine = ti < TB && t < p.T && col < cols;
  const int nq = p.q != nullptr ? p.Hq : 0;
  const int heads = nq + p.Hkv * (p.v != nullptr ? 2 : 1);

  auto source = [&](int h) -> const __nv_bfloat16* {
    if (h < nq) return p.q + t * p.qs[0] + h * p.qs[1];
    h -= nq;
    if (h < p.Hkv) return p.k + t * p.ks[0] + h * p.ks[1];
    return p.v + t * p.vs[0] + (h - p.Hkv) * p.vs[1];
  };
  C c;
  c.place(col, p.turn);
  typename C::Ch a[kAhead], bb[kAhead];
  if (mine) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (h0 + u * HS < heads) c.load(source(h0 + u * HS), a[u], bb[u]);
  }
  // Sequence of each of the block's tokens: how many sequences end at or
  // before it, by one parallel pass over the ends.
  marks[tid] = 0;
  __syncthreads();
  int before = 0;
  for (int j0 = 0; j0 < p.B; j0 += kThreadsRope) {
    const int end = j0 + tid < p.B ? p.cu_seqlens[j0 + tid + 1] : 0x7fffffff;
    if (end > t0 && end < t0 + TB) atomicAdd(&marks[end - t0], 1);
    before += __syncthreads_count(end <= t0);
  }
  // Position and place of each of them; row -1: a token of no sequence (or a refused step's).
  const int here = min(TB, p.T - t0);
  if (tid < here) {
    int b = before;
    for (int i = 1; i <= tid; ++i) b += marks[i];
    const int tt = t0 + tid;
    row[tid] = -1;
    pos[tid] = 0;
    page[tid] = -1;
    if (b < p.B && tt >= p.cu_seqlens[b] && (p.refused == nullptr || *p.refused == 0)) {
      const long slot = static_cast<long>(p.seq_lens[b]) - (p.cu_seqlens[b + 1] - tt);
      pos[tid] = p.pos != nullptr ? p.pos[tt] : static_cast<int>(slot);
      row[tid] = static_cast<int>(slot & (kTile - 1));
      if (slot >= 0 && slot < static_cast<long>(p.max_pages) * kTile) {
        const int pg = p.page_table[static_cast<long>(b) * p.max_pages + slot / kTile];
        if (pg >= 0 && pg < p.num_pages) page[tid] = pg;
      }
    }
  }
  __syncthreads();
  fill_table<C>(table, p.turn, pos, here, blockIdx.y * width, width);
  __syncthreads();
  if (!mine || row[ti] < 0) return;
  const bool in_cache = page[ti] >= 0;
  const long page_row = (static_cast<long>(page[ti]) * p.Hkv * kTile + row[ti]) * p.d;
  const long head_stride = static_cast<long>(kTile) * p.d;
  c.angles(table, ti, cw, width);
  for (int h = h0;;) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      int hh = h + u * HS;
      if (hh < heads) {
        if (hh < nq) {
          c.turn(a[u], bb[u]);
          c.store(p.q_out + t * p.qos[0] + hh * p.qos[1], a[u], bb[u]);
        } else if (in_cache) {
          hh -= nq;
          if (hh < p.Hkv) {
            c.turn(a[u], bb[u]);
            c.store(p.k_pages + page_row + hh * head_stride, a[u], bb[u]);
          } else {
            c.store(p.v_pages + page_row + (hh - p.Hkv) * head_stride, a[u], bb[u]);
          }
        }
      }
    }
    h += kAhead * HS;
    if (h >= heads) break;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (h + u * HS < heads) c.load(source(h + u * HS), a[u], bb[u]);
  }
}

// How a launch of `tokens` tokens x `heads` heads x `cols` columns is cut.
// HS, the threads that share a token's column, is what fills the GPU once
// (152 SMs of 2048 threads), at most a thread per head: a thread with many
// heads keeps loads in flight from batch to batch, one with few pays the
// block's two barriers and the angles for them.  Measured on 8192 tokens x 48
// heads of 128: HS = 6, 35 us; 11, 45 us; 20, 55 us; 3, 35 us.
struct Cut {
  int width, passes, HS, TB;
  unsigned blocks;
};
Cut cut_of(long tokens, int heads, int cols) {
  Cut c;
  c.passes = (cols + kThreadsRope - 1) / kThreadsRope;
  c.width = (cols + c.passes - 1) / c.passes;
  long hs = (152l * 2048 + tokens * cols - 1) / (tokens * cols);
  if (hs > heads) hs = heads;
  if (hs > kThreadsRope / c.width) hs = kThreadsRope / c.width;
  c.HS = static_cast<int>(hs);
  c.TB = kThreadsRope / (c.width * c.HS);
  c.blocks = static_cast<unsigned>((tokens + c.TB - 1) / c.TB);
  return c;
}

template <bool VEC, bool ADJ>
int columns(const RopeTurn& t, int d, bool in_place) {
  using C = Column<VEC, ADJ>;
  return C::turning(t.rot) + (in_place ? 0 : (d - t.rot) / C::kN);
}

template <bool VEC, bool ADJ>
cudaError_t rope_impl(const RopeParams& p, cudaStream_t st) {
  const int cols = columns<VEC, ADJ>(p.turn, p.d, p.x == p.out);
  const long tokens = static_cast<long>(p.B) * p.L;
  if (tokens == 0 || p.H == 0 || cols == 0) return cudaSuccess;
  if (tokens > 0x7fffffffL) return cudaErrorInvalidConfiguration;
  const Cut c = cut_of(tokens, p.H, cols);
  rope_kernel<VEC, ADJ><<<dim3(c.blocks, c.passes), kThreadsRope, 0, st>>>(p, cols, c.width, c.HS, c.TB);
  return cudaGetLastError();
}

template <bool VEC, bool ADJ>
cudaError_t append_impl(const AppendParams& p, cudaStream_t st) {
  const int cols = columns<VEC, ADJ>(p.turn, p.d, false);
  if (p.T == 0) return cudaSuccess;
  const int heads = (p.q != nullptr ? p.Hq : 0) + p.Hkv * (p.v != nullptr ? 2 : 1);
  const Cut c = cut_of(p.T, heads, cols);
  rope_append_kernel<VEC, ADJ><<<dim3(c.blocks, c.passes), kThreadsRope, 0, st>>>(p, cols, c.width, c.HS, c.TB);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool vec, cudaStream_t st) {
  if (vec) return p.turn.interleaved ? rope_impl<true, true>(p, st) : rope_impl<true, false>(p, st);
  return p.turn.interleaved ? rope_impl<false, true>(p, st) : rope_impl<false, false>(p, st);
}

cudaError_t launch_rope_append(const AppendParams& p, bool vec, cudaStream_t st) {
  if (vec)
    return p.turn.interleaved ? append_impl<true, true>(p, st) : append_impl<true, false>(p, st);
  return p.turn.interleaved ? append_impl<false, true>(p, st) : append_impl<false, false>(p, st);
}

}  // namespace ssattn

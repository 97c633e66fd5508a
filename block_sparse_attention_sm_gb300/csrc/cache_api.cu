// C-ABI entry points around the paged cache: rotary positions, the write of
// new tokens, attention of a chunk of new tokens, and the pages' bookkeeping.
// Argument validation and launches; include/ssattn.h has each call's contract.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <memory>
#include <new>

#include "api.cuh"
#include "chunk_paged.cuh"
#include "pages.cuh"
#include "rope.cuh"

namespace ssattn {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
bool all8(const long* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] % 8 != 0) return false;
  return true;
}

ss_status of(cudaError_t e) { return e == cudaSuccess ? SS_OK : SS_ERR_CUDA; }

// The rotation's own arguments; `vec`: its entries lie in whole 16-byte words.
ss_status turn_of(RopeTurn* t, const double* inv_freq, int rot, int off, int interleaved, float factor,
                  int inverse, int d, bool* vec) {
  if (rot < 0 || rot % 2 != 0 || off < 0 || rot > d || off > d - rot || !std::isfinite(factor))
    return SS_ERR_INVALID_ARG;
  if (rot > 0 && (inv_freq == nullptr || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0))
    return SS_ERR_INVALID_ARG;
  *t = RopeTurn{inv_freq, rot, off, interleaved ? 1 : 0, factor, inverse ? -1.f : 1.f};
  *vec = d % 8 == 0 && off % 8 == 0 && rot % (interleaved ? 8 : 16) == 0;
  return SS_OK;
}

constexpr int kMaxRopeWidth = 1 << 16;
// Rows and tokens are counted in 32 bits, a block's or a thread's share ahead.
constexpr long kMaxRopeCount = 1l << 30;

// Rows of d entries at these strides lie apart: each axis, from the smallest
// stride on, steps over everything that the axes before it reach.
bool rows_apart(const int64_t* stride, const int* size, int n, int d) {
  __int128 reach = d;
  bool used[3] = {false, false, false};
  for (int k = 0; k < n; ++k) {
    int next = -1;
    for (int i = 0; i < n; ++i)
      if (!used[i] && (next < 0 || stride[i] < stride[next])) next = i;
    used[next] = true;
    if (size[next] < 2) continue;
    if (stride[next] < reach) return false;
    reach += static_cast<__int128>(stride[next]) * (size[next] - 1);
  }
  return true;
}

// Memory of bf16 elements: up to four axes (stride, size), the contiguous one among them.
struct Span {
  struct Axis {
    __int128 stride, size;
  };
  const void* at;
  int n;
  Axis axis[4];
};
Span span(const void* at, std::initializer_list<Span::Axis> axes) {
  Span s{at, 0, {}};
  for (const Span::Axis& a : axes) {
    if (a.size < 2 || a.stride == 0) continue;
    int i = s.n++;
    for (; i > 0 && s.axis[i - 1].stride < a.stride; --i) s.axis[i] = s.axis[i - 1];
    s.axis[i] = a;  // (largest stride first)
  }
  return s;
}

// Whether two spans, the first `gap` elements in front of which the other
// starts, share elements.  Axis by axis from the largest stride: only those
// index differences k matter at which what is left of both comes together.
// Exact where the strides are the same (parts of one tensor); where more than
// a few k remain it answers true.
bool meet(__int128 gap, const Span::Axis* x, int nx, const Span::Axis* y, int ny) {
  __int128 ex = 1, ey = 1;  // how far each reaches
  for (int i = 0; i < nx; ++i) ex += x[i].stride * (x[i].size - 1);
  for (int i = 0; i < ny; ++i) ey += y[i].stride * (y[i].size - 1);
  if (gap >= ey || gap + ex <= 0) return false;
  if (nx == 0 && ny == 0) return true;
  const __int128 s = nx == 0 || (ny > 0 && y->stride > x->stride) ? y->stride : x->stride;
  __int128 cx = 1, cy = 1;
  if (nx > 0 && x->stride == s) cx = x->size, ex -= s * (cx - 1), ++x, --nx;
  if (ny > 0 && y->stride == s) cy = y->size, ey -= s * (cy - 1), ++y, --ny;
  const auto floor_div = [](__int128 a, __int128 b) { return a / b - (a % b < 0 ? 1 : 0); };
  __int128 lo = floor_div(-ex - gap, s) + 1, hi = floor_div(ey - gap - 1, s);
  if (lo < 1 - cy) lo = 1 - cy;
  if (hi > cx - 1) hi = cx - 1;
  if (hi - lo >= 4) return true;
  for (__int128 k = lo; k <= hi; ++k)
    if (meet(gap + k * s, x, nx, y, ny)) return true;
  return false;
}
bool meet(const Span& a, const Span& b) {
  if (a.at == nullptr || b.at == nullptr) return false;
  const __int128 gap = (static_cast<__int128>(reinterpret_cast<uintptr_t>(a.at)) - reinterpret_cast<uintptr_t>(b.at)) / 2;
  return meet(gap, a.axis, a.n, b.axis, b.n);
}

}  // namespace
}  // namespace ssattn

using namespace ssattn;

extern "C" {

ss_status ss_rope(const void* x, void* out, int B, int H, int L, int d, int64_t x_batch_stride,
                  int64_t x_head_stride, int64_t x_token_stride, int64_t out_batch_stride,
                  int64_t out_head_stride, int64_t out_token_stride, const int32_t* positions,
                  int64_t position_stride, const double* inv_freq, int rot_dim, int rot_offset,
                  int interleaved, int inverse, float attn_factor, void* stream) {
  if (B < 0 || H < 0 || L < 0 || d < 1 || rot_dim < 2 || position_stride < 0) return SS_ERR_INVALID_ARG;
  if (d > kMaxRopeWidth) return SS_ERR_UNSUPPORTED;
  RopeParams p{};
  bool vec = false;
  ss_status st = turn_of(&p.turn, inv_freq, rot_dim, rot_offset, interleaved, attn_factor, inverse, d, &vec);
  if (st != SS_OK) return st;
  if (B == 0 || H == 0 || L == 0) return SS_OK;
  const int64_t xs[3] = {x_batch_stride, x_head_stride, x_token_stride},
                os[3] = {out_batch_stride, out_head_stride, out_token_stride};
  const int size[3] = {B, H, L};
  for (int i = 0; i < 3; ++i) {
    p.xs[i] = xs[i];
    p.os[i] = os[i];
    if (xs[i] < 0 || os[i] < 0 || (x == out && size[i] > 1 && xs[i] != os[i])) return SS_ERR_INVALID_ARG;
  }
  // Rows of the output must not overlap; the input's may (a broadcast axis).
  if (!rows_apart(os, size, 3, d)) return SS_ERR_INVALID_ARG;
  if (H > kMaxRopeCount || static_cast<long>(B) * L > kMaxRopeCount) return SS_ERR_UNSUPPORTED;
  if (x == nullptr || out == nullptr || positions == nullptr || !aligned2(x) || !aligned2(out) ||
      !aligned4(positions))
    return SS_ERR_INVALID_ARG;
  const auto rows = [&](const void* at, const long* s) {
    return span(at, {{s[0], B}, {s[1], H}, {s[2], L}, {1, d}});
  };
  if (x != out && meet(rows(out, p.os), rows(x, p.xs))) return SS_ERR_INVALID_ARG;
  if ((st = check_device()) != SS_OK) return st;
  vec = vec && aligned16(x) && aligned16(out) && all8(p.xs, 3) && all8(p.os, 3);
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.pos = positions;
  p.pos_stride = position_stride;
  p.B = B;
  p.H = H;
  p.L = L;
  p.d = d;
  return of(launch_rope(p, vec, static_cast<cudaStream_t>(stream)));
}

ss_status ss_rope_append_paged_ex(const void* q, void* q_out, const void* k, const void* v,
                                  int64_t q_token_stride, int64_t q_head_stride, int64_t q_out_token_stride,
                                  int64_t q_out_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                                  int64_t v_token_stride, int64_t v_head_stride, int T, int B, int Hq,
                                  int Hkv, int d, const int32_t* cu_seqlens, const int32_t* seq_lens,
                                  const int32_t* positions, const double* inv_freq, int rot_dim,
                                  int rot_offset, int interleaved, float attn_factor, void* k_pages,
                                  void* v_pages, const int32_t* page_table, int num_pages, int max_pages,
                                  const int32_t* refused, void* stream) {
  if (T < 0 || B < 1 || Hkv < 1 || d < 1 || (q != nullptr && Hq < 1) || num_pages < 1 || max_pages < 1)
    return SS_ERR_INVALID_ARG;
  if (d > kMaxRopeWidth) return SS_ERR_UNSUPPORTED;
  AppendParams p{};
  bool vec = false;
  ss_status st = turn_of(&p.turn, inv_freq, rot_dim, rot_offset, interleaved, attn_factor, 0, d, &vec);
  if (st != SS_OK) return st;
  if (T == 0) return SS_OK;
  if (k == nullptr || k_pages == nullptr || cu_seqlens == nullptr || seq_lens == nullptr ||
      page_table == nullptr || (q != nullptr && q_out == nullptr) || (v != nullptr && v_pages == nullptr))
    return SS_ERR_INVALID_ARG;
  if (!aligned2(q) || !aligned2(q_out) || !aligned2(k) || !aligned2(v) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !aligned4(cu_seqlens) || !aligned4(seq_lens) || !aligned4(positions) ||
      !aligned4(page_table) || !aligned4(refused))
    return SS_ERR_INVALID_ARG;
  if (static_cast<long>(max_pages) * kTile > 0x7fffffffL) return SS_ERR_INVALID_ARG;
  const int64_t strides[4][2] = {{q_token_stride, q_head_stride},
                                 {q_out_token_stride, q_out_head_stride},
                                 {k_token_stride, k_head_stride},
                                 {v_token_stride, v_head_stride}};
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = q != nullptr ? strides[0][i] : 0;
    p.qos[i] = q != nullptr ? strides[1][i] : 0;
    p.ks[i] = strides[2][i];
    p.vs[i] = v != nullptr ? strides[3][i] : 0;
    if (p.qs[i] < 0 || p.ks[i] < 0 || p.vs[i] < 0) return SS_ERR_INVALID_ARG;
    if (q != nullptr && (p.qos[i] < 0 || (q == q_out && (i == 0 ? T : Hq) > 1 && p.qs[i] != p.qos[i])))
      return SS_ERR_INVALID_ARG;
  }
  const int q_size[2] = {T, Hq};
  if (q != nullptr && (!rows_apart(p.qos, q_size, 2, d) || q_out == k || q_out == v)) return SS_ERR_INVALID_ARG;
  if (T > kMaxRopeCount || Hq + 2l * Hkv > kMaxRopeCount) return SS_ERR_UNSUPPORTED;
  {  // what is written (q_out, the pools) lies apart from what is read, but for q turned in place
    const __int128 pool = static_cast<__int128>(num_pages) * Hkv * kTile * d;
    const auto rows = [&](const void* at, const long* s, int heads) {
      return span(at, {{s[0], T}, {s[1], heads}, {1, d}});
    };
    const Span in[3] = {rows(q, p.qs, Hq), rows(k, p.ks, Hkv), rows(v, p.vs, Hkv)};
    const Span to[3] = {rows(q != nullptr ? q_out : nullptr, p.qos, Hq), span(k_pages, {{1, pool}}),
                        span(v != nullptr ? v_pages : nullptr, {{1, pool}})};
    for (int i = 0; i < 3; ++i)
      for (int j = 0; j < 3; ++j)
        if (meet(to[i], in[j]) && !(i == 0 && j == 0 && q == q_out)) return SS_ERR_INVALID_ARG;
    if (meet(to[0], to[1]) || meet(to[0], to[2]) || meet(to[1], to[2])) return SS_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != SS_OK) return st;
  vec = vec && aligned16(q) && aligned16(q_out) && aligned16(k) && aligned16(v) && all8(p.ks, 2) &&
        (q == nullptr || (all8(p.qs, 2) && all8(p.qos, 2))) && (v == nullptr || all8(p.vs, 2));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  p.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  p.cu_seqlens = cu_seqlens;
  p.seq_lens = seq_lens;
  p.pos = positions;
  p.page_table = page_table;
  p.refused = refused;
  p.T = T;
  p.B = B;
  p.Hq = q != nullptr ? Hq : 0;
  p.Hkv = Hkv;
  p.d = d;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  return of(launch_rope_append(p, vec, static_cast<cudaStream_t>(stream)));
}

ss_status ss_rope_append_paged(const void* q, void* q_out, const void* k, const void* v,
                               int64_t q_token_stride, int64_t q_head_stride, int64_t q_out_token_stride,
                               int64_t q_out_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                               int64_t v_token_stride, int64_t v_head_stride, int T, int B, int Hq,
                               int Hkv, int d, const int32_t* cu_seqlens, const int32_t* seq_lens,
                               const int32_t* positions, const double* inv_freq, int rot_dim,
                               int rot_offset, int interleaved, float attn_factor, void* k_pages,
                               void* v_pages, const int32_t* page_table, int num_pages, int max_pages,
                               void* stream) {
  return ss_rope_append_paged_ex(q, q_out, k, v, q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride,
                                 k_token_stride, k_head_stride, v_token_stride, v_head_stride, T, B, Hq, Hkv, d,
                                 cu_seqlens, seq_lens, positions, inv_freq, rot_dim, rot_offset, interleaved,
                                 attn_factor, k_pages, v_pages, page_table, num_pages, max_pages, nullptr, stream);
}

ss_status ss_rope_frequencies(double* out, int rot_dim, double base, ss_rope_scaling scaling,
                              double factor, int original_length, double lo, double hi,
                              float* attn_factor_out) {
  if (out == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
    return SS_ERR_INVALID_ARG;
  if (scaling != SS_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return SS_ERR_INVALID_ARG;
  const bool ramped = scaling == SS_ROPE_YARN || scaling == SS_ROPE_WAVELENGTH;
  if (ramped && (original_length < 1 || !(lo > 0.0) || !(hi > lo) || !std::isfinite(hi)))
    return SS_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  double b = base;
  if (scaling == SS_ROPE_BASE) {
    if (rot_dim < 4) return SS_ERR_INVALID_ARG;
    b = base * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  }
  double first = 0.0, last = 0.0;  // SS_ROPE_YARN: the ramp's ends, in pairs
  if (scaling == SS_ROPE_YARN) {
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(original_length / (turns * two_pi)) / (2.0 * std::log(base));
    };
    first = std::fmax(0.0, std::floor(pair_of(hi)));
    last = std::fmin(rot_dim - 1.0, std::ceil(pair_of(lo)));
    if (last - first < 1e-3) last = first + 1e-3;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double w = std::pow(b, -2.0 * i / rot_dim);
    double keep = 1.0;  // share of the unscaled frequency
    switch (scaling) {
      case SS_ROPE_PLAIN:
      case SS_ROPE_BASE: break;
      case SS_ROPE_LINEAR: keep = 0.0; break;
      case SS_ROPE_YARN: keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - first) / (last - first))); break;
      case SS_ROPE_WAVELENGTH:
        keep = std::fmin(1.0, std::fmax(0.0, (original_length * w / two_pi - lo) / (hi - lo)));
        break;
      default: return SS_ERR_INVALID_ARG;
    }
    out[i] = scaling == SS_ROPE_PLAIN ? w : w * keep + w / factor * (1.0 - keep);
  }
  if (attn_factor_out != nullptr)
    *attn_factor_out = scaling == SS_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return SS_OK;
}

size_t ss_attn_chunk_paged_units(int T, int B, int Hq, int Hkv) {
  if (T < 0 || B < 1 || Hkv < 1 || Hq < Hkv) return 0;
  const int G = Hq / Hkv;
  if (G > kTile) return 0;
  return 2 * static_cast<size_t>(chunk_slots(T, B, kTile / G)) * Hkv;
}

size_t ss_attn_chunk_paged_workspace_size(int T, int B, int Hq, int Hkv, int max_pages, int d,
                                          int num_kv_splits) {
  if (num_kv_splits <= 1 || T < 1 || B < 1 || Hkv < 1 || Hq < Hkv || Hq / Hkv > kTile || max_pages < 1 ||
      d < 1)
    return 0;
  const int parts = chunk_parts(chunk_slots(T, B, kTile / (Hq / Hkv)) * Hkv, num_kv_splits, max_pages);
  return parts == 1 ? 0 : static_cast<size_t>(parts) * T * Hq * (d + 2) * sizeof(float);
}

size_t ss_attn_chunk_paged_workspace_bound(int T, int Hq, int Hkv, int max_pages, int d, int num_kv_splits) {
  if (num_kv_splits <= 1 || T < 1 || Hkv < 1 || Hq < Hkv || Hq / Hkv > kTile || max_pages < 1 || d < 1) return 0;
  // The most parts are made for one sequence; fewer, the more places its tokens
  // take.  Of the steps with the same places, the longest needs the most.
  const long pair = 2 * (kTile / (Hq / Hkv));
  size_t most = 0;
  for (long places = 1;; ++places) {
    const int parts = chunk_parts(places * Hkv, num_kv_splits, max_pages);
    const long tokens = std::min<long>(T, places * pair - 1);
    if (parts > 1) most = std::max(most, static_cast<size_t>(parts) * tokens);
    if (parts == 1 || tokens == T) return most * Hq * (d + 2) * sizeof(float);
  }
}

ss_status ss_attn_chunk_paged(const void* q, int64_t q_token_stride, const void* k_pages,
                              const void* v_pages, const int32_t* page_table, const int32_t* cu_seqlens,
                              const int32_t* seq_lens, void* o, int T, int B, int Hq, int Hkv,
                              int num_pages, int max_pages, int d, float scale, int causal,
                              float lambda_a, int num_kv_splits, uint32_t* skip_counts, void* workspace,
                              size_t workspace_bytes, const ss_debug_opts* dbg, void* stream) {
  if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_pages < 1 || max_pages < 1 ||
      num_kv_splits < 1 || !(scale > 0.f) || !std::isfinite(scale) || !(lambda_a >= 0.f) ||
      !std::isfinite(lambda_a))
    return SS_ERR_INVALID_ARG;
  if (dbg != nullptr && (dbg->count_only || dbg->fault_inject || dbg->vote_chunk_tiles || dbg->prefill_kernel))
    return SS_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return SS_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G > kTile) return SS_ERR_UNSUPPORTED;
  if ((T > 0 && (q == nullptr || o == nullptr)) || k_pages == nullptr || v_pages == nullptr ||
      page_table == nullptr || cu_seqlens == nullptr || seq_lens == nullptr)
    return SS_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(Hq) * d, stride = q_token_stride != 0 ? q_token_stride : row;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) ||
      !aligned4(page_table) || !aligned4(cu_seqlens) || !aligned4(seq_lens) || stride < row || stride % 8 != 0)
    return SS_ERR_INVALID_ARG;
  const long tpb = kTile / G, slots = chunk_slots(T, B, tpb);
  if (static_cast<long>(max_pages) * kTile > 0x7fffffffL || T > 0x7fffffff - 2 * kTile ||
      static_cast<long>(num_pages + 1L) * Hkv > 0x7fffffffL ||
      slots > 0x3fffffffL || Hkv > 65535 || 2 * slots * Hkv > 0x7fffffffL ||
      static_cast<long>(T) * Hq > 8 * 0x7fffffffL || stride >= (1LL << 38))
    return SS_ERR_INVALID_ARG;
  const size_t need = ss_attn_chunk_paged_workspace_size(T, B, Hq, Hkv, max_pages, d, num_kv_splits);
  if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
    return SS_ERR_WORKSPACE;
  {  // the queries of a block are read again by other clusters, the pools throughout
    const Span out = span(o, {{1, static_cast<long>(T) * row}});
    const long pool = static_cast<long>(num_pages) * Hkv * kTile * d;
    if (T > 0 && (meet(out, span(q, {{stride, T}, {1, row}})) || meet(out, span(k_pages, {{1, pool}})) ||
                  meet(out, span(v_pages, {{1, pool}}))))
      return SS_ERR_INVALID_ARG;
  }
  const bool outputs = skip_counts != nullptr || (dbg != nullptr && (dbg->skip_mask || dbg->vote_margin));
  if (T == 0 && !outputs) return SS_OK;
  ss_status st = check_device();
  if (st != SS_OK) return st;
  if (T == 0) {  // no tokens: every unit's outputs are those of one without tokens
    const size_t units = 2 * static_cast<size_t>(slots) * Hkv, seen = units * max_pages;
    const auto s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (skip_counts != nullptr) e = cudaMemsetAsync(skip_counts, 0, units * sizeof(uint32_t), s);
    if (e == cudaSuccess && dbg != nullptr && dbg->skip_mask != nullptr)
      e = cudaMemsetAsync(dbg->skip_mask, 2, seen, s);
    if (e == cudaSuccess && dbg != nullptr && dbg->vote_margin != nullptr)
      e = cudaMemsetAsync(dbg->vote_margin, 0xff, seen * sizeof(float), s);  // (all ones: a NaN)
    return of(e);
  }

  CUtensorMap tq, tk, tv;
  const long blocks = static_cast<long>(num_pages) * Hkv;
  if (!make_map(&tk, k_pages, d, kTile, blocks, kTile / 2) || !make_map(&tv, v_pages, d, kTile, blocks))
    return SS_ERR_CUDA;
  {  // q as [T][Hkv][G][d]; a box is 64 entries of a row block
    auto fn = encode_fn();
    if (fn == nullptr) return SS_ERR_CUDA;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(G),
                                static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(G) * d * 2,
                                   static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(tpb)};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    if (fn(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return SS_ERR_CUDA;
  }
  ChunkParams p{};
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.tpb = static_cast<int>(tpb);
  p.slots = static_cast<int>(slots);
  p.S = num_kv_splits < max_pages ? num_kv_splits : max_pages;  // (a range has a tile or more)
  p.parts = chunk_parts(slots * Hkv, num_kv_splits, max_pages);
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.causal = causal ? 1 : 0;
  p.scale = scale;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.lambda_a = lambda_a;
  p.cu_seqlens = cu_seqlens;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.o = static_cast<__nv_bfloat16*>(o);
  if (p.parts > 1) {
    const size_t rows = static_cast<size_t>(p.parts) * T * Hq;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + rows * d);
  }
  p.counts = skip_counts;
  p.mask = dbg != nullptr ? dbg->skip_mask : nullptr;
  p.margin = dbg != nullptr ? dbg->vote_margin : nullptr;
  p.status = status_ptr();
  const bool vote = lambda_a > 0.f || p.mask != nullptr || p.margin != nullptr;
  return of(launch_chunk_paged(d, vote, tq, tk, tv, p, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- pages

size_t ss_pages_workspace_size(int num_pages, int num_rows, int n) {
  if (num_pages < 0 || num_rows < 0 || n < 0) return 0;
  return pages_workspace(num_pages, num_rows, n);
}

static ss_status check_state(const int32_t* refs, int num_pages, const int32_t* table, int num_rows,
                             int max_pages, const int32_t* lens) {
  if (refs == nullptr || table == nullptr || lens == nullptr || num_pages < 1 || num_rows < 1 ||
      max_pages < 1 || static_cast<long>(max_pages) * kTile > 0x7fffffffL || !aligned16(refs) ||
      !aligned4(table) || !aligned4(lens))
    return SS_ERR_INVALID_ARG;
  return SS_OK;
}

// Bytes of a pool, or more than any memory where that is too many to count.
static size_t pool_bytes_of(size_t page_bytes, int num_pages) {
  return page_bytes > SIZE_MAX / num_pages ? SIZE_MAX : page_bytes * num_pages;
}

static ss_status check_pools(void* const* pools, int num_pools, size_t page_bytes) {
  if (num_pools < 0 || (num_pools > 0 && pools == nullptr) || page_bytes == 0 || page_bytes % 16 != 0 ||
      page_bytes > (static_cast<size_t>(1) << 34))
    return SS_ERR_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i)
    if (pools[i] == nullptr || !aligned16(pools[i])) return SS_ERR_INVALID_ARG;
  return SS_OK;
}

namespace {
// An array that a call is given; `written`: that it writes.
struct Range {
  const void* at;
  size_t bytes;
  bool written;
  bool meets(const Range& r) const {
    const auto a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(r.at);
    return bytes > 0 && r.bytes > 0 && (a <= b ? b - a < bytes : a - b < r.bytes);
  }
};
Range reads(const int32_t* p, long n) { return {p, p != nullptr ? 4 * static_cast<size_t>(n) : 0, false}; }
Range writes(const int32_t* p, long n) { return {p, p != nullptr ? 4 * static_cast<size_t>(n) : 0, true}; }

// Nothing that a call writes may overlap anything else of it.  A pool listed
// twice is copied twice, to the same bytes; different pools lie apart.
ss_status check_apart(std::initializer_list<Range> arrays, void* const* pools = nullptr, int num_pools = 0,
                      size_t pool_bytes = 0) {
  for (const Range* a = arrays.begin(); a != arrays.end(); ++a)
    for (const Range* b = a + 1; b != arrays.end(); ++b)
      if ((a->written || b->written) && a->meets(*b)) return SS_ERR_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i)
    for (const Range& a : arrays)
      if (a.meets({pools[i], pool_bytes, true})) return SS_ERR_INVALID_ARG;
  // Pools one behind the other, the usual order, take one pass, others are sorted.
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  bool in_order = true;
  for (int i = 1; i < num_pools; ++i)
    in_order = in_order && at(pools[i]) > at(pools[i - 1]) && at(pools[i]) - at(pools[i - 1]) >= pool_bytes;
  if (in_order) return SS_OK;
  std::unique_ptr<uintptr_t[]> sorted(new (std::nothrow) uintptr_t[num_pools]);
  if (sorted == nullptr) return SS_ERR_CUDA;
  for (int i = 0; i < num_pools; ++i) sorted[i] = at(pools[i]);
  std::sort(sorted.get(), sorted.get() + num_pools);
  for (int i = 1; i < num_pools; ++i)
    if (sorted[i] != sorted[i - 1] && sorted[i] - sorted[i - 1] < pool_bytes) return SS_ERR_INVALID_ARG;
  return SS_OK;
}
}  // namespace

static ss_status check_workspace(const void* ws, size_t bytes, int num_pages, int num_rows, int n) {
  return ws == nullptr || !aligned16(ws) || bytes < pages_workspace(num_pages, num_rows, n)
             ? SS_ERR_WORKSPACE
             : SS_OK;
}

ss_status ss_pages_reserve(int32_t* page_refs, int num_pages, int32_t* page_table, int num_rows,
                           int max_pages, int32_t* seq_lens, const int32_t* rows, const int32_t* add,
                           int n, int32_t* result, void* workspace, size_t workspace_bytes,
                           void* stream) {
  ss_status st = check_state(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens);
  if (st != SS_OK) return st;
  if (n < 0 || (n > 0 && add == nullptr) || !aligned4(rows) || !aligned4(add) || !aligned4(result) ||
      (rows == nullptr && n > num_rows))
    return SS_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, num_pages, num_rows, n)) != SS_OK) return st;
  const long entries = static_cast<long>(num_rows) * max_pages;
  st = check_apart({writes(page_refs, num_pages), writes(page_table, entries), writes(seq_lens, num_rows),
                    writes(result, 1), {workspace, pages_workspace(num_pages, num_rows, n), true}, reads(rows, n),
                    reads(add, n)});
  if (st != SS_OK || (st = check_device()) != SS_OK) return st;
  const PageState s{page_refs, page_table, seq_lens, num_pages, num_rows, max_pages};
  return of(launch_pages_reserve(s, rows, add, n, result, workspace, static_cast<cudaStream_t>(stream)));
}

ss_status ss_pages_free(int32_t* page_refs, int num_pages, int32_t* page_table, int num_rows,
                        int max_pages, int32_t* seq_lens, const int32_t* rows, int n, void* stream) {
  ss_status st = check_state(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens);
  if (st != SS_OK) return st;
  if (n < 0 || (n > 0 && rows == nullptr) || !aligned4(rows)) return SS_ERR_INVALID_ARG;
  const long entries = static_cast<long>(num_rows) * max_pages;
  st = check_apart({writes(page_refs, num_pages), writes(page_table, entries), writes(seq_lens, num_rows),
                    reads(rows, n)});
  if (st != SS_OK || (st = check_device()) != SS_OK) return st;
  const PageState s{page_refs, page_table, seq_lens, num_pages, num_rows, max_pages};
  return of(launch_pages_free(s, rows, n, static_cast<cudaStream_t>(stream)));
}

ss_status ss_pages_fork(void* const* pools, int num_pools, size_t page_bytes, int32_t* page_refs,
                        int num_pages, int32_t* page_table, int num_rows, int max_pages,
                        int32_t* seq_lens, const int32_t* src_rows, const int32_t* dst_rows, int n,
                        int32_t* result, void* workspace, size_t workspace_bytes, void* stream) {
  ss_status st = check_state(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens);
  if (st != SS_OK || (st = check_pools(pools, num_pools, page_bytes)) != SS_OK) return st;
  if (n < 0 || (n > 0 && (src_rows == nullptr || dst_rows == nullptr)) || !aligned4(src_rows) ||
      !aligned4(dst_rows) || !aligned4(result))
    return SS_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, num_pages, num_rows, n)) != SS_OK) return st;
  const long entries = static_cast<long>(num_rows) * max_pages;
  st = check_apart({writes(page_refs, num_pages), writes(page_table, entries), writes(seq_lens, num_rows),
                    writes(result, 1), {workspace, pages_workspace(num_pages, num_rows, n), true},
                    reads(src_rows, n), reads(dst_rows, n)},
                   pools, num_pools, pool_bytes_of(page_bytes, num_pages));
  if (st != SS_OK || (st = check_device()) != SS_OK) return st;
  const PageState s{page_refs, page_table, seq_lens, num_pages, num_rows, max_pages};
  return of(launch_pages_fork(pools, num_pools, page_bytes, s, src_rows, dst_rows, n, result, workspace,
                              static_cast<cudaStream_t>(stream)));
}

ss_status ss_pages_copy(void* const* pools, int num_pools, size_t page_bytes, int num_pages,
                        const int32_t* src, const int32_t* dst, int n, int32_t* result, void* workspace,
                        size_t workspace_bytes, void* stream) {
  ss_status st = check_pools(pools, num_pools, page_bytes);
  if (st != SS_OK) return st;
  if (num_pools < 1 || num_pages < 1 || n < 0 || (n > 0 && (src == nullptr || dst == nullptr)) ||
      !aligned4(src) || !aligned4(dst) || !aligned4(result))
    return SS_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, num_pages, 0, n)) != SS_OK) return st;
  st = check_apart({writes(result, 1), {workspace, pages_workspace(num_pages, 0, n), true}, reads(src, n),
                    reads(dst, n)},
                   pools, num_pools, pool_bytes_of(page_bytes, num_pages));
  if (st != SS_OK || (st = check_device()) != SS_OK) return st;
  return of(launch_pages_copy(pools, num_pools, page_bytes, num_pages, src, dst, n, result, workspace,
                              static_cast<cudaStream_t>(stream)));
}

ss_status ss_pages_compact(void* const* pools, int num_pools, size_t page_bytes, int32_t* page_refs,
                           int num_pages, int32_t* page_table, int num_rows, int max_pages,
                           const int32_t* seq_lens, int32_t* out_refs, int32_t* out_table, int32_t* live,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int32_t* lens = const_cast<int32_t*>(seq_lens);
  ss_status st = check_state(page_refs, num_pages, page_table, num_rows, max_pages, lens);
  if (st != SS_OK || (st = check_pools(pools, num_pools, page_bytes)) != SS_OK) return st;
  if (out_refs == nullptr) out_refs = page_refs;
  if (out_table == nullptr) out_table = page_table;
  if (!aligned4(out_refs) || !aligned4(out_table) || !aligned4(live)) return SS_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, num_pages, num_rows, 0)) != SS_OK) return st;
  const long entries = static_cast<long>(num_rows) * max_pages;
  st = check_apart({writes(out_refs, num_pages), writes(out_table, entries),
                    reads(out_refs != page_refs ? page_refs : nullptr, num_pages),
                    reads(out_table != page_table ? page_table : nullptr, entries), reads(lens, num_rows),
                    writes(live, 1), {workspace, pages_workspace(num_pages, num_rows, 0), true}},
                   pools, num_pools, pool_bytes_of(page_bytes, num_pages));
  if (st != SS_OK || (st = check_device()) != SS_OK) return st;
  const PageState s{page_refs, page_table, lens, num_pages, num_rows, max_pages};
  return of(launch_pages_compact(pools, num_pools, page_bytes, s, out_refs, out_table, live, workspace,
                                 static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

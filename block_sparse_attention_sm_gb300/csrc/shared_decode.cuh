// Declarations of the decode over shared pages, shared with the C-ABI layer.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace ssattn {

// A plan of shared pages, int32 words.  The sequences in the order of their
// tables' pages ([kPlanHead, kPlanHead + B)), then 2 B nodes of kNodeWords:
// node i < B is what the sequence at place i has to itself, node B + i the
// pages shared by a run of places (empty: not used); then for each place the
// kPlanLevels nodes above it, from the deepest up (-1: none).
constexpr int kPlanHead = 8;    // words: B, max_pages, a mark
constexpr int kPlanMark = 0x504c414e;
constexpr int kNodeWords = 4;   // first place, places, first tile, end tile
constexpr int kPlanLevels = 7;  // shared nodes above a sequence at most (bounds the partial results)
constexpr int kPlanMaxB = 8192;
constexpr int kSharedMaxB = 32768;  // sequences of a decode without a plan (their sums fit shared memory)

__host__ __device__ constexpr size_t plan_words(long B) { return kPlanHead + B + 2 * B * kNodeWords + B * kPlanLevels; }

cudaError_t launch_prefix_plan(const int32_t* table, const int32_t* lens, int B, int max_pages,
                               int32_t* plan, cudaStream_t st);

// The results of one level (its own tiles, or a node above) of a (place, KV head): those of head g in rows row + g,
// row + g + second, and the same a CTA's rows on, and so on; `count` of them (second = 0: one a CTA).
struct Parts {
  long long row;
  int second, count;
};

struct SharedParams {
  int B, Hq, Hkv, G;
  uint32_t inv_g;          // floor(2^32 / G) + 1 (G > 1): r / G of a row r is the product's upper half
  int num_pages, max_pages;
  int ctas;                // CTAs of the attention kernel
  float scale_log2;
  const __nv_bfloat16* q;  // [B][Hq][d], rows of heads q_stride apart
  long q_stride;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* plan;     // nullable
  __nv_bfloat16* o;        // [B][Hq][d]
  float* part_o;           // [part_rows][d] unnormalised partial outputs
  float2* part_ml;         // [part_rows] (reference maximum in exp2 units, sum)
  long part_rows;
  Parts* parts;            // [B][Hkv][1 + kPlanLevels], without a plan [B][Hkv]
  float* lse;              // [B][Hq] log2 of the softmax's denominator (weights only)
  float* scores;           // [B][Hq][max_pages][128] (weights only)
  float* weights;          // [B][Hkv][max_pages * 128], nullable
  uint32_t* status;
};

// Tiles over all sequences and KV heads that a table may have room for: their cost (3 a tile and 3 an item at
// most, and as much again for each level of shared nodes at most) is counted in 32 bits.
constexpr long kMaxSharedTiles = 1l << 29, kMaxPlannedTiles = 1l << 26;

// Workspace: sizes and where its arrays lie.
struct SharedSpace {
  size_t part_o, part_ml, parts, lse, scores, bytes;
  long part_rows;
};
SharedSpace shared_space(int B, int Hq, int Hkv, int max_pages, int d, bool plan, bool weights);
int shared_ctas(int B, int Hq, int Hkv, int max_pages);

cudaError_t launch_shared_decode(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const SharedParams& p, cudaStream_t st);

}  // namespace ssattn

// Declarations of the chunk attention over the paged cache, shared with the C-ABI layer.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace ssattn {

struct ChunkParams {
  int T, B, Hq, Hkv, G;    // packed new tokens, sequences, heads, Hq / Hkv
  int tpb;                 // tokens of a row block: 128 / G
  int slots;               // places for pairs of row blocks (see chunk_slots)
  int S;                   // ranges of the vote that a sequence's tiles are cut into
  int parts;               // parts that the tiles are dealt to (<= S)
  int num_pages, max_pages;
  int causal;
  float scale, scale_log2, lambda_a;
  const int32_t* cu_seqlens;
  const int32_t* seq_lens;
  const int32_t* page_table;
  __nv_bfloat16* o;        // [T][Hq][d]
  float* part_o;           // parts > 1: [parts][T * Hq][d] unnormalised outputs
  float2* part_ml;         // parts > 1: [parts][T * Hq] (reference maximum in exp2 units, sum)
  uint32_t* counts;
  uint8_t* mask;
  float* margin;
  uint32_t* status;
};

// Pairs of row blocks are numbered without knowing the sequences' lengths on
// the host: with P = 2 * tpb tokens a pair, sequence b's pairs start at place
// floor(cu[b] / P) + b, which leaves room for ceil(n_b / P) of them before the
// next sequence's (floor((c + n) / P) + 1 - floor(c / P) >= ceil(n / P)).
__host__ __device__ constexpr long chunk_slots(long T, long B, long tpb) {
  return T / (2 * tpb) + B;
}

// How many parts to deal the tiles of `pairs` pairs of row blocks (over all KV heads) to.
int chunk_parts(long pairs, int S, int max_pages);

cudaError_t launch_chunk_paged(int d, bool vote, const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, const ChunkParams& p, cudaStream_t st);

}  // namespace ssattn

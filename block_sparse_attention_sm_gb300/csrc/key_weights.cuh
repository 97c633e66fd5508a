// Declarations of the record of attention weights by new tokens, shared with the C-ABI layer.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace ssattn {

struct KeyWeightsParams {
  int T, B, Hq, Hkv, G;
  int tpb;                 // tokens of a row block: 128 / G
  uint64_t tpb_inverse;    // ceil(2^64 / tpb), where that is below 2^64
  int num_pages, max_pages;
  int causal;
  int ctas;
  int whole;               // items are not cut
  float scale_log2;
  const int32_t* cu_seqlens;
  const int32_t* seq_lens;
  const int32_t* page_table;
  float* weights;          // [B][Hkv][max_pages * 128]
  float* lse;              // [Hkv][places][2][128] -log2 of the rows' denominators, by place of their pair of blocks
  long places;
  float2* part_ml;         // [ctas][2][256] results of split items: rows' (m, l)
  float* part_w;           // [ctas][2][256] keys' sums
  struct Split* split;     // [ctas] the item that a CTA begins and does not end
  uint32_t* status;
};

// What the CTAs behind have to add to the item that this one begins.
struct Split {
  int valid, b, kvh, pair;
  int left, per;  // steps left to the CTAs behind, steps of a CTA's share
};

// Pairs of row blocks are numbered as in the chunk attention: those of sequence b start at floor(cu[b] / (2 tpb)) + b.
__host__ __device__ constexpr long key_weights_places(long T, long B, long tpb) { return T / (2 * tpb) + B; }

struct KeyWeightsSpace {
  size_t lse, part_ml, part_w, split, bytes;
};
KeyWeightsSpace key_weights_space(int T, int B, int Hq, int Hkv);

cudaError_t launch_key_weights(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                               const KeyWeightsParams& p, cudaStream_t st);

}  // namespace ssattn

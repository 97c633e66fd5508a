// Declarations of the rotary-position kernels, shared with the C-ABI layer.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace ssattn {

// Strides are in elements; the innermost axis is contiguous.
struct RopeTurn {
  const double* inv_freq;  // [rot / 2] radians per position
  int rot, off;            // rotated entries [off, off + rot) of each row
  int interleaved;         // pairs (2i, 2i + 1); otherwise (i, i + rot / 2)
  float factor;            // of cosines and sines
  float sign;              // +1, or -1 for the transposed rotation
};

struct RopeParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  long xs[3], os[3];        // (batch, head, token)
  const int32_t* pos;
  long pos_stride;          // between batch entries; 0: one row of positions for all
  int B, H, L, d;
  RopeTurn turn;
};

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;  // q, v nullable
  __nv_bfloat16 *q_out, *k_pages, *v_pages;
  long qs[2], qos[2], ks[2], vs[2];  // (token, head)
  const int32_t *cu_seqlens, *seq_lens, *pos, *page_table;  // pos nullable
  const int32_t* refused;  // nullable: nothing is done where it is not 0
  int T, B, Hq, Hkv, d, num_pages, max_pages;
  RopeTurn turn;
};

cudaError_t launch_rope(const RopeParams& p, bool vec, cudaStream_t st);
cudaError_t launch_rope_append(const AppendParams& p, bool vec, cudaStream_t st);

}  // namespace ssattn

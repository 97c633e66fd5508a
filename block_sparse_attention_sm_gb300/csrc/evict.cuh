// Declarations of the cache's eviction by accumulated weight, shared with the C-ABI layer.
#pragma once
#include "pages.cuh"

namespace ssattn {

struct EvictArgs {
  PageState s;              // refs and table are replaced by out_*, lens by out_lens
  void* const* pools;       // host: num_layers x per_layer device addresses
  float* const* weights;    // host: [num_layers] device addresses, [num_rows][Hkv][max_pages * 128]
  float* const* out_weights;
  int num_layers, per_layer, Hkv;
  size_t page_bytes;
  const int32_t* rows;      // nullable
  const int32_t* keep;
  int n, recent;
  int32_t* out_refs;
  int32_t* out_table;
  int32_t* out_lens;
  int32_t* result;
};

size_t evict_workspace(int num_pages, int num_rows, int max_pages, int n, int Hkv, int num_layers, int per_layer);

cudaError_t launch_pages_evict(const EvictArgs& a, void* ws, cudaStream_t st);

}  // namespace ssattn

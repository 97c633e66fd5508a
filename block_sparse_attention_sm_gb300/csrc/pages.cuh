// Declarations of the page-bookkeeping kernels, shared with the C-ABI layer.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ssattn {

constexpr int kMaxPools = 64;  // pools per copy launch (their addresses are kernel parameters)

// The cache's bookkeeping: how many sequences hold each page (0: free), each
// sequence's pages, and its length.
struct PageState {
  int32_t* refs;   // [num_pages]
  int32_t* table;  // [num_rows][max_pages]
  int32_t* lens;   // [num_rows]
  int num_pages, num_rows, max_pages;
};

struct PagePools {
  unsigned char* base[kMaxPools];
  int count;
  size_t page_bytes;
};

size_t pages_workspace(int num_pages, int num_rows, int n);

cudaError_t launch_pages_reserve(const PageState& s, const int32_t* rows, const int32_t* add, int n,
                                 int32_t* result, void* ws, cudaStream_t st);
cudaError_t launch_pages_free(const PageState& s, const int32_t* rows, int n, cudaStream_t st);
cudaError_t launch_pages_fork(void* const* pools, int num_pools, size_t page_bytes,
                              const PageState& s, const int32_t* src, const int32_t* dst, int n,
                              int32_t* result, void* ws, cudaStream_t st);
cudaError_t launch_pages_copy(void* const* pools, int num_pools, size_t page_bytes, int num_pages,
                              const int32_t* src, const int32_t* dst, int n, int32_t* result,
                              void* ws, cudaStream_t st);
cudaError_t launch_pages_compact(void* const* pools, int num_pools, size_t page_bytes,
                                 const PageState& s, int32_t* out_refs, int32_t* out_table,
                                 int32_t* live, void* ws, cudaStream_t st);

}  // namespace ssattn

// Helpers of the C-ABI layer, shared by its translation units.
#pragma once
#include <cudaTypedefs.h>

#include "common.cuh"

namespace ssattn {

// Device address of the status word for the current device (cached).
uint32_t* status_ptr();

bool aligned16(const void* ptr);

// The current device must be sm_103 (GB300); cached per device ordinal.
ss_status check_device();

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// 3-D view [BH][L][d] of a bf16 tensor, 64 x box_rows boxes, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int d, int L, long BH, int box_rows = kTile);

}  // namespace ssattn

// ops.h - shared by the operators beside the fused block (rows.cu, linear.cu):
// argument checks and element sizes (not public).
#pragma once

#include <cuda_runtime.h>

#include <initializer_list>

#include "beam_moe.h"

namespace beam {

inline size_t dtype_bytes(int32_t dtype) { return dtype == BEAM_MOE_FP32 ? 4 : 2; }

inline beam_moe_status cuda_status(cudaError_t e) {
  return e == cudaSuccess ? BEAM_MOE_OK : BEAM_MOE_ERR_CUDA;
}

// Required pointers are not NULL, and none is off a 16-byte boundary.
inline beam_moe_status check_ops_ptrs(std::initializer_list<const void*> required,
                                      std::initializer_list<const void*> optional) {
  for (const void* p : required)
    if (!p) return BEAM_MOE_ERR_INVALID_ARG;
  for (const void* p : required)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return BEAM_MOE_ERR_ALIGNMENT;
  for (const void* p : optional)
    if (p && (reinterpret_cast<uintptr_t>(p) & 15u)) return BEAM_MOE_ERR_ALIGNMENT;
  return BEAM_MOE_OK;
}

}  // namespace beam

// Helpers shared by the translation units of the C ABI's device calls.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// PKV_ERR_CUDA with the CUDA error's text.
pkv_status cuda_fail(cudaError_t e, const char *where);

// SMs of the current device (-1: cannot be queried).
int sm_count();

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link); NULL if unavailable.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Add to the calling thread's launch count (pkv_launch_count).
void add_launches(int64_t delta);

}  // namespace pkv

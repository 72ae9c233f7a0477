// What the C ABI's source files share.
#pragma once

#include <cudaTypedefs.h>

#include <cstdint>

#include "common.cuh"

namespace mqa {

// Records e for mqa_last_cuda_error on this thread; returns MQA_ERR_CUDA.
mqa_status api_cuda_fail(cudaError_t e);

// cuTensorMapEncodeTiled of the loaded driver, or null.
PFN_cuTensorMapEncodeTiled_v12000 api_encode_tiled();

// SMs of the current device, or -1.
int api_sm_count();

// Whether the test hooks (mqa_decode_testing.h) may run.
bool api_test_hooks();

inline bool api_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace mqa

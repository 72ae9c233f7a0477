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

// A cap of logits: none, or far enough from the ends of the fp32 range that it
// and its reciprocal are normal numbers.
inline bool api_softcap_ok(float cap) { return cap == 0.f || (cap >= 0x1p-20f && cap <= 0x1p60f); }

// Whether nx bytes at x and ny bytes at y overlap.
inline bool api_overlap(const void* x, size_t nx, const void* y, size_t ny) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return x && y && nx > 0 && ny > 0 && a < b + ny && b < a + nx;
}

// Bytes that a call reads or writes (none where p is null).
struct ApiSpan {
    const void* p;
    size_t n;
};
// Whether one of the spans that a call writes lies on another of its spans.  (A span that is written in place is among
// the written ones alone.)
template <int W, int R>
bool api_clash(const ApiSpan (&writes)[W], const ApiSpan (&reads)[R]) {
    for (int i = 0; i < W; ++i) {
        for (int j = i + 1; j < W; ++j)
            if (api_overlap(writes[i].p, writes[i].n, writes[j].p, writes[j].n)) return true;
        for (const ApiSpan& r : reads)
            if (api_overlap(writes[i].p, writes[i].n, r.p, r.n)) return true;
    }
    return false;
}

}  // namespace mqa

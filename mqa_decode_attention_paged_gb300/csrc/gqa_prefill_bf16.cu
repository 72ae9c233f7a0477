// Prompt attention over caches in bf16 (gqa_prefill_kernel.cuh).
#include "gqa_prefill_kernel.cuh"

namespace mqa {

cudaError_t pre_stage1_bf16(const PreArgs& a, int D, cudaStream_t stream) { return pre::dispatch<kWinBf16, false>(a, D, stream); }

}  // namespace mqa

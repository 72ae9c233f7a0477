// Prompt attention over caches of int8 codes (gqa_prefill_kernel.cuh).
#include "gqa_prefill_kernel.cuh"

namespace mqa {

cudaError_t pre_stage1_int8(const PreArgs& a, int D, cudaStream_t stream) { return pre::dispatch<kWinInt8, true>(a, D, stream); }

}  // namespace mqa

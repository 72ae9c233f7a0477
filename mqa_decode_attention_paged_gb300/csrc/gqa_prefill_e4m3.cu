// Prompt attention over caches of e4m3 codes (gqa_prefill_kernel.cuh).
#include "gqa_prefill_kernel.cuh"

namespace mqa {

cudaError_t pre_stage1_e4m3(const PreArgs& a, int D, cudaStream_t stream) { return pre::dispatch<kWinE4m3, false>(a, D, stream); }

}  // namespace mqa

// Prompt attention over caches of e4m3 codes with block scales (gqa_prefill_kernel.cuh).
#include "gqa_prefill_kernel.cuh"

namespace mqa {

cudaError_t pre_stage1_e4m3_block(const PreArgs& a, int D, cudaStream_t stream) { return pre::dispatch<kWinE4m3, true>(a, D, stream); }

}  // namespace mqa

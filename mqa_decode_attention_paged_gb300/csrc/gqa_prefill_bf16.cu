// Prompt attention over bf16 caches (gqa_prefill_kernel.cuh).
#include "gqa_prefill_kernel.cuh"

namespace mqa {

cudaError_t pre_stage1_bf16(const PreArgs& a, int D, cudaStream_t stream) { return pre::dispatch<kWinBf16>(a, D, stream); }

}  // namespace mqa

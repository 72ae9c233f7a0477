// Prompt attention over bf16 caches (gqa_prefill_kernel.cuh).
#include "gqa_prefill_kernel.cuh"

namespace mqa {

cudaError_t pre_stage1_bf16(const PreArgs& a, int D, bool shaped, cudaStream_t stream) {
    return shaped ? pre::dispatch<kWinBf16, true>(a, D, stream) : pre::dispatch<kWinBf16, false>(a, D, stream);
}

}  // namespace mqa

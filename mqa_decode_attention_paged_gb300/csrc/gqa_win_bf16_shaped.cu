// GQA decode with shaped logits, stage 1, bf16 caches (gqa_win_kernel.cuh).
#include "gqa_win_kernel.cuh"

namespace mqa {

cudaError_t win_shaped_bf16(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    return win::dispatch<kWinBf16, true>(a, D, grid, stream);
}

}  // namespace mqa

// GQA decode with shaped logits, stage 1, e4m3 caches (gqa_win_kernel.cuh).
#include "gqa_win_kernel.cuh"

namespace mqa {

cudaError_t win_shaped_e4m3(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    return win::dispatch<kWinE4m3, true>(a, D, grid, stream);
}

}  // namespace mqa

// Windowed / block-scaled GQA decode, stage 1, e4m3 caches (gqa_win_kernel.cuh).
#include "gqa_win_kernel.cuh"

namespace mqa {

cudaError_t win_stage1_e4m3(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    return win::dispatch<kWinE4m3>(a, D, grid, stream);
}

}  // namespace mqa

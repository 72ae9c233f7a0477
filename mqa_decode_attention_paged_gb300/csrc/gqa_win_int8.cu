// Windowed / block-scaled GQA decode, stage 1, int8 caches (gqa_win_kernel.cuh).
#include "gqa_win_kernel.cuh"

namespace mqa {

cudaError_t win_stage1_int8(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    return win::dispatch<kWinInt8>(a, D, grid, stream);
}

}  // namespace mqa

// Windowed / block-scaled GQA decode, stage 1, bf16 caches (gqa_win_kernel.cuh).
#include "gqa_win_kernel.cuh"

namespace mqa {

cudaError_t win_stage1_bf16(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    return win::dispatch<kWinBf16, false>(a, D, grid, stream);
}

}  // namespace mqa

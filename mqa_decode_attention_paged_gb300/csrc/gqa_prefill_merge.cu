// Prompt attention, stage 2: the partials of each cut (cell, head) merged (out =
// sum_s w_s O_s / sum_s w_s l_s, w_s = 2^{m_s - max m}; ascending thread blocks,
// so the result is reproducible).
//
// Bound by reading the partials, 4 D bytes a row and piece, mostly from L2.  The
// block of thread block c's begun (cell, head) finds its pieces among the blocks
// after c; a warp takes four of the 32 rows in turn.  3 to 8 us in a warm graph.
#include "gqa_prefill.cuh"

namespace mqa {
namespace {

constexpr int kMaxGrid = 256;
constexpr int kRowsPerBlock = 32;

template <int D>
__global__ void __launch_bounds__(256) pre_merge_kernel(const __grid_constant__ PreArgs a) {
    __shared__ int state[kMaxGrid];
    __shared__ int slots[kMaxGrid];
    __shared__ int count;
    __shared__ float weight[8][kMaxGrid];
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();  // stage 1 is done
    const int4 meta = a.ws_meta[2 * c];
    const int first = static_cast<int>(blockIdx.y) * kRowsPerBlock;
    if (meta.x != 1 || first % kPreTile >= a.tile_rows || first / kPreTile * a.tile_tok >= meta.w) return;
    const int h = a.ws_meta[2 * c + 1].x;
    for (int d = c + 1 + threadIdx.x; d < a.grid; d += blockDim.x) state[d] = a.ws_meta[2 * d].y;
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        slots[n++] = 2 * c + 1;
        for (int d = c + 1; d < a.grid; ++d) {
            if (state[d] == 3) continue;
            if (state[d] != 1 && state[d] != 2) break;  // (a block that gave up: undefined rows, and the status says so)
            slots[n++] = 2 * d;
            if (state[d] == 1) break;
        }
        count = n;
    }
    __syncthreads();
    const int np = count;
    constexpr int V = D / 32;
    for (int k = 0; k < kRowsPerBlock / 8; ++k) {
        const int row = first + k * 8 + warp, i = row / kPreTile, r = row % kPreTile;
        const int tk = a.grp_div(r), token = i * a.tile_tok + tk;
        if (r >= a.tile_rows || token >= meta.w) continue;  // (the warp's rows end together)
        float mx = -INFINITY;
        for (int p = lane; p < np; p += 32)
            mx = fmaxf(mx, __ldg(a.ws_ml + 2 * (static_cast<long long>(slots[p]) * kPreSlotRows + row)));
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float ref = mx == -INFINITY ? 0.f : mx;
        float l = 0.f;
        __syncwarp();
        for (int p = lane; p < np; p += 32) {
            const float2 ml = __ldg(reinterpret_cast<const float2*>(a.ws_ml) + static_cast<long long>(slots[p]) * kPreSlotRows + row);
            const float w = ex2(ml.x - ref);
            weight[warp][p] = w;
            l += ml.y * w;
        }
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        __syncwarp();
        float acc[V] = {};
        constexpr int kInFlight = 8;
        for (int p0 = 0; p0 < np; p0 += kInFlight) {
            float x[kInFlight][V];
#pragma unroll
            for (int e = 0; e < kInFlight; ++e) {
                const bool have = p0 + e < np && weight[warp][p0 + e] != 0.f;
                const float* o = a.ws_o + (static_cast<long long>(slots[have ? p0 + e : 0]) * kPreSlotRows + row) * D + lane * V;
                if constexpr (V == 4) {
                    const float4 y = have ? __ldg(reinterpret_cast<const float4*>(o)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[e][0] = y.x;
                    x[e][1] = y.y;
                    x[e][2] = y.z;
                    x[e][3] = y.w;
                } else {
                    const float2 y = have ? __ldg(reinterpret_cast<const float2*>(o)) : make_float2(0.f, 0.f);
                    x[e][0] = y.x;
                    x[e][1] = y.y;
                }
            }
#pragma unroll
            for (int e = 0; e < kInFlight; ++e) {
                const float w = p0 + e < np ? weight[warp][p0 + e] : 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[e][v], acc[v]);
            }
        }
        const float f = l == 0.f ? 0.f : 1.f / l;
        const long long orow = static_cast<long long>(meta.z + token) * a.Hq + h * a.grp + (r - tk * a.grp);
        if constexpr (V == 4)
            *reinterpret_cast<uint2*>(a.out + orow * D + lane * V) =
                make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
        else
            *reinterpret_cast<uint32_t*>(a.out + orow * D + lane * V) = pack_bf16x2(acc[0] * f, acc[1] * f);
        if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
    }
}

}  // namespace

cudaError_t pre_merge(const PreArgs& a, int D, cudaStream_t stream) {
    static_assert(kPreSlotRows % kRowsPerBlock == 0 && kPreTile % kRowsPerBlock == 0, "row groups");
    const dim3 grid(a.grid - 1, kPreSlotRows / kRowsPerBlock);  // (the last thread block begins nothing that it does not end)
    if (a.grid < 2) return cudaSuccess;
    return D == 128 ? launch_with_pdl(pre_merge_kernel<128>, grid, dim3(256), 0, stream, a)
                    : launch_with_pdl(pre_merge_kernel<64>, grid, dim3(256), 0, stream, a);
}

}  // namespace mqa

// Windowed / block-scaled GQA decode, stage 2: the partials of each row merged
// by LogSumExp (out = sum_s w_s O_s / sum_s w_s, w_s = e^{lse_s - max lse},
// lse = max + ln sum w; ascending units, so the result is reproducible).
//
// Bound by the latency of its few loads: a row has np partials of D fp32
// values.  One warp per row where a row has few partials, a block of 8 warps
// per row (each takes every eighth partial, then a sum through shared memory)
// where few rows are cut into many; the host picks by the mean number of
// partials.  Stage 1 left each request's first and last unit in the
// workspace; a request of one unit was written by it and is skipped.
#include "gqa_win.cuh"

namespace mqa {
namespace {

constexpr int kWarps = 8;
constexpr int kInFlight = 8;  // partials of a row whose loads are issued together

template <int V>
struct Vec;
template <>
struct Vec<4> {
    using T = float4;
};
template <>
struct Vec<2> {
    using T = float2;
};

// WPR: warps per row (1 or kWarps).
template <int D, int WPR>
__global__ void __launch_bounds__(32 * kWarps) win_merge_kernel(const __grid_constant__ WinArgs a) {
    constexpr int V = D / 32;
    using VecT = typename Vec<V>::T;
    __shared__ float part[WPR == 1 ? 1 : kWarps][D + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int v = blockIdx.x;
    const int b = a.rb_div(v), r = v - b * a.rb;
    const int item = WPR == 1 ? static_cast<int>(blockIdx.y) * kWarps + warp : static_cast<int>(blockIdx.y);
    const int kh = item / a.rbn, jr = item - kh * a.rbn;
    const int R = r * a.rbn + jr;
    pdl_wait();  // stage 1 is done (every warp waits, so that this grid ends after it)
    const int2 units = a.ws_units[v];
    const int gf = units.x, np = units.y - units.x + 1;
    if (np == 1 || kh >= a.Hkv || R >= a.rows) return;
    // (a unit that gave up may have left this entry unwritten, or partials: the
    // row is then undefined, and the status word says so)
    if (units.x < 0 || units.y < units.x || units.y >= a.units) return;
    const int i = a.grp_div(R);
    const long long orow = (static_cast<long long>(b) * a.q_len + i) * a.Hq + kh * a.grp + (R - i * a.grp);
    __nv_bfloat16* out = a.out + orow * D + V * lane;

    const long long step = static_cast<long long>(a.Hkv) * a.rbn;  // rows per slot
    const long long first = (static_cast<long long>(gf + v) * a.Hkv + kh) * a.rbn + jr;
    // the first partials' loads are in flight before their weights are known
    float x[kInFlight][V], ls[kInFlight];
    auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int s = s0 + u * WPR;
            ls[u] = -INFINITY;
            if (s < np) {
                ls[u] = a.ws_lse[first + s * step];
                *reinterpret_cast<VecT*>(x[u]) =
                    __ldcs(reinterpret_cast<const VecT*>(a.ws_o + (first + s * step) * D + V * lane));
            }
        }
    };
    const int start = WPR == 1 ? 0 : warp;
    load(start);
    float m = -INFINITY;
    for (int s = lane; s < np; s += 32) m = fmaxf(m, a.ws_lse[first + s * step]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mu = m == -INFINITY ? 0.f : m;  // a NaN partial has a NaN weight, and so has the row

    float acc[V] = {};
    float wsum = 0.f;
    for (int s0 = start; s0 < np; s0 += kInFlight * WPR) {
        if (s0 > start) load(s0);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const float w = __expf(ls[u] - mu);
            wsum += w;
            if (w != 0.f)
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += w * x[u][k];
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int k = 0; k < V; ++k) part[warp][V * lane + k] = acc[k];
        if (lane == 0) part[warp][D] = wsum;
        __syncthreads();
        if (warp > 0) return;
        for (int s = 1; s < kWarps; ++s) {
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += part[s][V * lane + k];
            wsum += part[s][D];
        }
    }
    const float inv = wsum != 0.f ? 1.f / wsum : 0.f;  // 0: no visible key
#pragma unroll
    for (int k = 0; k < V; k += 2)
        *reinterpret_cast<uint32_t*>(out + k) = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
    if (a.lse && lane == 0) a.lse[orow] = wsum != 0.f ? mu + logf(wsum) : -INFINITY;
}

template <int D, int WPR>
cudaError_t launch(const WinArgs& a, cudaStream_t stream) {
    const int items = a.Hkv * a.rbn;
    return launch_with_pdl(win_merge_kernel<D, WPR>,
                           dim3(a.batch * a.rb, WPR == 1 ? (items + kWarps - 1) / kWarps : items),
                           dim3(32 * kWarps), 0, stream, a);
}

}  // namespace

cudaError_t win_merge(const WinArgs& a, int D, cudaStream_t stream) {
    // a row is summed from about units / (batch * rb) + 1 partials: 10 of them
    // in 4096 rows take 21 us with a block per row, 8 us with a warp
    const bool many = a.units > 16 * a.batch * a.rb;
    if (D == 128) return many ? launch<128, kWarps>(a, stream) : launch<128, 1>(a, stream);
    return many ? launch<64, kWarps>(a, stream) : launch<64, 1>(a, stream);
}
}  // namespace mqa

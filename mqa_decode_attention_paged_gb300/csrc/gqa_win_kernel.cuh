// Stage 1 of windowed / block-scaled GQA paged decode (see gqa_win.cuh for the
// plan).  For query row r and key t of its KV head
//   x_t = scale * s_k <q_r, K_t>,  out_r = sum_t e^{x_t - lse_r} s_v V_t,
//   lse_r = ln sum_t e^{x_t}
// with s_k, s_v the scales of the token block and head (1 for bf16).
//
// What bounds it: the bytes of the visible keys and values, read once (a
// row block of up to 24 rows does 12 multiply-adds per byte of bf16 cache and
// twice that per 8-bit byte, far below the tensor rate), and, with an 8-bit
// cache, the instructions that widen the codes.
//
// One thread block = up to 8 warps, two blocks per SM (128 registers a
// thread; over bf16 one reads at full rate, and that is what is launched where
// requests are cut), or one where more than 8 rows meet head size 128
// (accumulators and Q of 16 rows alone are 96 registers) or more than 16 head
// size 64.  Warp w takes KV head w % Hkv and part w / Hkv of every tile, and
// feeds itself: it keeps a ring of slots in shared memory, copies its own
// head's K rows and then V rows of a tile into it with tensor copies (16 or 32
// token rows of one head, 128-byte or 64-byte swizzle: ldmatrix over eight
// tokens is free of bank conflicts and nothing is padded), and refills a slot
// as soon as it has read it.  There is no producer warp (whose registers
// would cost every thread 32) and no barrier between warps but a meeting
// every kMeet tiles, so that the heads of a token row are read near each other:
// a probe that only copies reads 6.9 TB/s with such per-head boxes and three
// 2 KB slots, but 3.9 TB/s where six slots let the warps drift apart (in this
// kernel 1, 2, 8 and 64 tiles between meetings are within 3 % of each other).
// Boxes are described 16 at a time, a lane each, across requests.
//
// Measured (batch of 256, lognormal lengths, 32/8 heads x 128, 16-token pages,
// e4m3 with a scale per page and head): 259 us, 6.4 TB/s of the 6.67 a copy
// reaches; 64 windows of 16384 tokens over bf16: 594 us, 7.2 TB/s (reads alone
// run faster than a copy).  Short windows are bound by the start (4.3 us until
// the copies are issued) and the merge; 9 to 16 rows per KV head by instructions
// (32 windows of 4096 over e4m3, 16 rows, head size 128: 69 us; with two blocks
// per SM, half the tokens per step and Q in shared memory it was 92 us and 730
// instructions per 16 tokens and head).  17 to 24 rows are one row block: 32
// windows of 2000, 20 rows, take 59 (bf16), 54 (e4m3) and 49 (int8) us; as two
// blocks of 16 and 4 rows bf16 took 95 and e4m3 73.
//   * Tokens are the MMA's M dimension: S^T = K Q^T (16 tokens x 8 rows),
//     O^T = V^T P^T (16 head dims x 8 rows); NHB row groups of 8.
//   * 8-bit codes stay codes in shared memory and are widened to f16 in
//     registers.  K: four consecutive codes of a token to a lane; Q has the
//     same order.  V: ldmatrix.trans over byte pairs gives a lane two head dims
//     of two tokens; byte permutes make the two f16 pairs, so accumulator rows
//     g and g + 8 are head dims 2g and 2g + 1.  (The warp-level e4m3 MMA is no
//     way around the widening of K: with Q in two e4m3 terms it took 399 us
//     where f16 took 342, on 256 requests of lognormal length.)
//   * Online softmax in base 2; the reference moves only when a logit exceeds
//     it by more than 8, which a warp vote finds without reductions.  Over
//     8-bit caches the numerators keep a reference of their own for x +
//     log2(s_v): the weights of P.V stay within the f16 range whatever the
//     scales' magnitude, and V is not rescaled.
//   * Masked keys: their logits are replaced by -inf, and at the edges of what
//     the rows see V rows of keys that none sees are cleared in the slot, so
//     stale or non-finite bytes never reach an accumulator (int8 codes are
//     always finite).  Where a key is seen by some rows only and a V value is
//     Inf or NaN, the rows are summed apart; where a V scale is, the numerators'
//     reference of the rows that see it becomes NaN, and the scale counts as 1
//     (the weight of a masked key would be e^{-inf + inf}).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "gqa_win.cuh"

namespace mqa {
namespace win {

constexpr int kMaxSlots = 4;
constexpr int kChunk = 16;  // boxes described together
constexpr int kDesc = 64;   // box descriptions kept per warp: at most three chunks are in use
constexpr int kMeet = 8;    // tiles between meetings of a block's warps
constexpr float kNone = -3e38f;  // reference before the first logit

template <int D, int KIND, int NHB>
struct Cfg {
    static constexpr int kElt = KIND == kWinBf16 ? 2 : 1;
    static constexpr int kLine = D * kElt >= 128 ? 128 : D * kElt;  // bytes of one swizzled line
    static constexpr int kPanels = D * kElt / kLine;
    static constexpr int kSteps = D / 16;
    static constexpr int kMT = win_mblocks(KIND, NHB, D);
    static constexpr int kTok = 16 * kMT;            // tokens of a warp's tile
    static constexpr int kSlot = kTok * D * kElt;    // bytes of a slot (one plane of it)
    // A lane hands its accumulators to another warp 16 at a time, or all at once
    // where eight full rings, four warps' buffers and 26 KB for the rest fit
    // (42 requests, 35 rows of one KV head, int8: 48 -> 42 us)
    static constexpr int kAll = 4 * NHB * kSteps, kTail = 6 * NHB;
    static constexpr bool kRoom = 8 * kMaxSlots * kSlot + 4 * (kAll + kTail) * 128 + 26 * 1024 <=
                                  228 * 1024 / win_ctas_per_sm(NHB, D);
    static constexpr int kHanded = kRoom ? kAll : 16;
    static constexpr int kExch = (kHanded + kTail) * 128;  // one warp's hand-over buffer
};

struct Layout {
    int exch, scales, desc, bars, cum, total;  // the warps' rings come first
};

template <int D, int KIND, int NHB>
__host__ __device__ inline Layout layout(int hkv, int ts, int nslots, int vb, int batch) {
    using C = Cfg<D, KIND, NHB>;
    const int nc = hkv * ts;
    Layout l;
    l.exch = nc * nslots * C::kSlot;
    l.scales = l.exch + (ts > 1 ? nc / 2 * C::kExch : 0);
    l.desc = l.scales + nc * kMaxSlots * 16;
    l.bars = l.desc + nc * kDesc * 16;
    l.cum = l.bars + nc * kMaxSlots * 8;
    l.total = l.cum + 4 * (vb + 2 + batch) + 1024;  // + alignment of the base
    return l;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Box of one head from cache row `row` on.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const void* tmap, int row, int head, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %2, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(0), "r"(row), "r"(head), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrive on `bar` (one of its expected arrivals) when this thread's earlier
// cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// d = a b + d, or a b if `first`, on 16-bit operands (bf16, else f16).  No
// memory is touched: the compiler may schedule it freely.
template <int KIND>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                    bool first = false) {
    const float c0 = first ? 0.f : d[0], c1 = first ? 0.f : d[1], c2 = first ? 0.f : d[2], c3 = first ? 0.f : d[3];
    if constexpr (KIND == kWinBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Transpose of an 8x8 matrix of 16-bit values in the MMA fragment layout.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }
// P is rounded to the cache's operand type: bf16 beside bf16 values, f16
// beside widened codes (the denominator sums the unrounded fp32 values).
template <int KIND>
__device__ __forceinline__ uint32_t p_pair(float lo, float hi) {
    return KIND == kWinBf16 ? pack_bf16x2(lo, hi) : f16_pair(lo, hi);
}
__device__ __forceinline__ uint32_t q_f16(uint32_t v) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
    return f16_pair(f.x, f.y);
}

// The two e4m3 codes in the low half of w as two f16 values (exact).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// Bytes `sel` of u (codes + 128) as two f16 values: 1024 + u is exact in the
// mantissa of 0x6400, minus 1152 gives the code.
__device__ __forceinline__ uint32_t int8_pair(uint32_t u, uint32_t sel) {
    return half2_bits(__hsub2(bits_half2(__byte_perm(u, 0x64646464u, sel)), bits_half2(0x64806480u)));
}
// Four codes -> the f16 pairs of bytes (0, 1) and (2, 3).
template <int KIND>
__device__ __forceinline__ uint2 widen_adjacent(uint32_t w) {
    if constexpr (KIND == kWinInt8) {
        const uint32_t u = w ^ 0x80808080u;
        return make_uint2(int8_pair(u, 0x4140), int8_pair(u, 0x4342));
    } else {
        return make_uint2(e4m3_pair(w), e4m3_pair(w >> 16));
    }
}
// Four codes -> the f16 pairs of bytes (0, 2) and (1, 3).
template <int KIND>
__device__ __forceinline__ uint2 widen_strided(uint32_t w) {
    if constexpr (KIND == kWinInt8) {
        const uint32_t u = w ^ 0x80808080u;
        return make_uint2(int8_pair(u, 0x4240), int8_pair(u, 0x4341));
    } else {
        return make_uint2(e4m3_pair(__byte_perm(w, 0u, 0x4420)), e4m3_pair(__byte_perm(w, 0u, 0x4431)));
    }
}

// Whether a word of V (two bf16 values or four e4m3 codes) holds an Inf or NaN.
template <int KIND>
__device__ __forceinline__ bool non_finite(uint32_t w) {
    if constexpr (KIND == kWinBf16) return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    const uint32_t x = w & 0x7f7f7f7fu;
    return (x & 0xffu) == 0x7fu || (x & 0xff00u) == 0x7f00u || (x & 0xff0000u) == 0x7f0000u ||
           (x & 0xff000000u) == 0x7f000000u;
}

// The rest of a wait that did not end at once.
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity); }

// cum[0 .. vb]: exclusive prefix of the virtual requests' tile counts, then the
// largest count; lens: clamped lengths.  Every thread of the block calls it;
// returns the total.
__device__ __forceinline__ int build_prefix(const WinArgs& a, int* cum, int* lens) {
    const int vb = a.batch * a.rb;
    for (int v = threadIdx.x; v < vb; v += blockDim.x) {
        const int b = a.rb == 1 ? v : a.rb_div(v), r = v - b * a.rb;
        const int n = win_len(a, b, a.status);
        if (r == 0) lens[b] = n;
        cum[v + 1] = win_visible(a, r, n).nt;
    }
    if (threadIdx.x == 0) cum[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        int running = 0, longest = 0;
        for (int base = 0; base < vb; base += 32) {
            const int i = base + static_cast<int>(threadIdx.x);
            int x = i < vb ? cum[i + 1] : 0;
            longest = max(longest, x);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o);
                if (static_cast<int>(threadIdx.x) >= o) x += u;
            }
            if (i < vb) cum[i + 1] = running + x;
            running += __shfl_sync(0xffffffffu, x, 31);
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (threadIdx.x == 0) cum[vb + 1] = longest;
    }
    __syncthreads();
    return cum[vb];
}

// A box of tokens: x first token, y its row of the K plane (-1: nothing to
// copy; the V plane is a page of rows further), z the virtual request and the
// flags below, w the index of its first K scale.
constexpr int kVMask = kWinMaxVirtual - 1;
constexpr int kFirst = 1 << 11, kLast = 1 << 12, kWhole = 1 << 13;  // of the tile in the unit's run of its request
// of the tile's 16-token blocks (up to four): holds a key that the rows see,
// and one that some row does not see
constexpr int kAct = 1 << 14, kEdge = 1 << 18, kBlocks = 15;
constexpr int kSteps2 = 22;  // bits 22 + 2j: scales from the box's first to that of its 16 tokens number j + 1

// MULTI: more than one query position per request.
template <int D, int KIND, int NHB, bool MULTI>
__global__ void __launch_bounds__(256, win_ctas_per_sm(NHB, D)) gqa_win_kernel(const __grid_constant__ WinArgs a) {
    using C = Cfg<D, KIND, NHB>;
    constexpr int MT = C::kMT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int Hkv = a.Hkv, TS = a.ts, NC = Hkv * TS, nslots = a.nslots;
    const int vb = a.batch * a.rb;
    const Layout lay = layout<D, KIND, NHB>(Hkv, TS, nslots, vb, a.batch);
    int* cum = reinterpret_cast<int*>(smem + lay.cum);
    int* lens = cum + vb + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / Hkv, kh = warp - sub * Hkv;
    const bool scaled = KIND != kWinBf16 && a.kv_scales != nullptr;
    const uint32_t ring = smem_u32(smem) + warp * nslots * C::kSlot;
    float* scale_s = reinterpret_cast<float*>(smem + lay.scales) + warp * kMaxSlots * 4;  // [slot][MMA block]
    int4* desc_s = reinterpret_cast<int4*>(smem + lay.desc) + warp * kDesc;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars) + warp * kMaxSlots;
    const int nb = C::kTok / a.box_tok;  // boxes of a warp's tile (1, 2 or 4)
    const int nb_log = nb >> 1;

    if (lane == 0) {
        if (warp == 0) prefetch_tmap(&a.tmap);
        // a fill: each box's bytes, and its scales
        for (int s = 0; s < nslots; ++s) mbar_init(&full[s], scaled ? 2 * nb : nb);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const int T = build_prefix(a, cum, lens);  // contains __syncthreads

    // this block's tiles [p0, p1)
    int p0, p1;
    const int U = a.units == 0 ? 0 : win_units(a, vb, T, cum[vb + 1]);
    if (U == 0) {  // a unit is a request
        p0 = cum[min(static_cast<int>(blockIdx.x), vb)];
        p1 = cum[min(static_cast<int>(blockIdx.x) + 1, vb)];
    } else {
        const int u = min(static_cast<int>(blockIdx.x), U);
        p0 = win_unit_start(T, U, u);
        p1 = win_unit_start(T, U, min(u + 1, U));
    }
    // virtual requests without a key: out = 0, lse = -inf
    for (int v = blockIdx.x; v < vb; v += gridDim.x) {
        if (cum[v + 1] > cum[v]) continue;
        const int b = a.rb_div(v), r0 = (v - b * a.rb) * a.rbn, rows = min(a.rows - r0, a.rbn);
        for (int i = threadIdx.x; i < Hkv * rows * (D / 8); i += blockDim.x) {
            const int h = i / (rows * (D / 8)), R = r0 + i / (D / 8) % rows, qi = R / a.grp;
            const long long orow = (static_cast<long long>(b) * a.q_len + qi) * a.Hq + h * a.grp + R - qi * a.grp;
            *reinterpret_cast<uint4*>(a.out + orow * D + i % (D / 8) * 8) = make_uint4(0u, 0u, 0u, 0u);
            if (a.lse && i % (D / 8) == 0) a.lse[orow] = -INFINITY;
        }
        if (a.units > 0 && threadIdx.x == 0) a.ws_units[v] = make_int2(0, 0);
    }

    // ---- copying.  Boxes are described kChunk at a time, a lane each (across
    // requests), in shared memory for the copies and for the reader: locate()
    // writes all but the block ids, and fetches those; complete() puts them in
    // when the chunk's turn comes, a chunk later.
    const int boxes = (p1 - p0) * nb;
    int located = 0, completed = 0;  // boxes
    int id = -1;                     // block id of box located - kChunk + lane; -2: not a block
    auto locate = [&]() {
        const int i = located + lane;
        int4 d = make_int4(0, 0, 0, 0);
        id = -1;
        if (lane < kChunk && i < boxes) {
            const int P = p0 + (i >> nb_log), k = i & (nb - 1);  // tile, box of it
            int lo = 0, hi = vb - 1;  // the last virtual request starting at or before P
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cum[mid] <= P)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int b = a.rb == 1 ? lo : a.rb_div(lo);
            const WinVis vis = win_visible(a, lo - b * a.rb, lens[b]);
            const int c0 = cum[lo], c1 = cum[lo + 1];
            d.x = (vis.tile(P - c0) << a.tt_log) + sub * C::kTok + k * a.box_tok;
            d.z = lo | (P == max(c0, p0) ? kFirst : 0) | (P + 1 == min(c1, p1) ? kLast : 0) |
                  (c0 >= p0 && c1 <= p1 ? kWhole : 0);
            const int page = a.page_div(d.x);
            d.y = d.x - page * a.page;
            if (scaled) d.w = a.scale_div(d.y);
            for (int m = 0; m < a.box_tok / 16; ++m) {
                const int t = d.x + 16 * m, bit = k * (a.box_tok / 16) + m;
                const bool act = t <= vis.p_last && (t + 15 > vis.p_first - a.window || t < a.sinks);
                const bool edge = !act || t + 15 > vis.p_first || (t + 15 >= a.sinks && t <= vis.p_last - a.window);
                d.z |= (act ? kAct << bit : 0) | (edge ? kEdge << bit : 0);
                if (scaled && m > 0) d.z |= (a.scale_div(d.y + 16 * m) - d.w) << (kSteps2 - 2 + 2 * m);
            }
            // only boxes with a visible key are read, and only their block ids
            if (d.z & (kBlocks * kAct)) {
                id = __ldg(a.block_table + static_cast<long long>(b) * a.max_blocks + page);
                if (id < 0 || id >= a.num_blocks) id = -2;
            }
        }
        if (lane < kChunk && i < boxes) {
            desc_s[i & (kDesc - 1)] = d;
            if (d.z & kFirst) {  // the request's query will be wanted soon
                const int v = d.z & kVMask, qb0 = a.rb == 1 ? v : a.rb_div(v);
                const char* q0 = reinterpret_cast<const char*>(
                    a.q + (static_cast<long long>(qb0) * a.q_len * a.Hq + kh * a.grp) * D);
                for (int o = 0; o < a.grp * D * 2; o += 128) prefetch_l2(q0 + o);
            }
        }
        located += kChunk;
    };
    auto complete = [&]() {
        const int i = completed + lane;
        int4 d = make_int4(0, -1, 0, 0);
        if (lane < kChunk && i < boxes) {
            d = desc_s[i & (kDesc - 1)];
            if (id == -2) report(a.status, MQA_ERR_DEVICE_CHECK);
            if (id < 0) {  // nothing to read: no block of it counts
                d.z = (d.z & ~(kBlocks * kAct)) | ((d.z & (kBlocks * kAct)) / kAct * kEdge);
                d.y = -1;
            } else {
                d.y += id * 2 * a.page;
                d.w = (id * 2 * a.scale_groups + d.w) * Hkv + kh;
            }
        }
        // every box of a tile carries the flags of all its blocks
        for (int s = 1; s < nb; s <<= 1)
            d.z |= __shfl_xor_sync(0xffffffffu, d.z, s) & (kBlocks * kAct | kBlocks * kEdge);
        if (lane < kChunk && i < boxes) desc_s[i & (kDesc - 1)] = d;
        __syncwarp();
        completed += kChunk;
    };
    const int loads = 2 * (p1 - p0);  // planes to copy: K, V, K, V ..
    int issued = 0, i_slot = 0;
    auto issue = [&]() {
        const int first = (issued >> 1) * nb, plane = issued & 1;
        if (lane < nb && static_cast<int>(blockIdx.x) != a.withhold) {
            const int4 d = desc_s[(first + lane) & (kDesc - 1)];
            const int bytes = C::kSlot >> nb_log;
            if (d.y >= 0) {
                mbar_arrive_expect_tx(&full[i_slot], bytes);
                tma_load_rows(ring + i_slot * C::kSlot + lane * bytes, &a.tmap, d.y + plane * a.page, kh,
                              &full[i_slot]);
                if (scaled) {
                    const float* sp = a.kv_scales + d.w + plane * (a.scale_groups * Hkv);
                    float* dst = scale_s + i_slot * 4 + (lane * MT >> nb_log);
                    cp_async_4(dst, sp);
#pragma unroll
                    for (int m = 1; m < MT; ++m)
                        if (16 * m < a.box_tok)
                            cp_async_4(dst + m, sp + ((d.z >> (kSteps2 - 2 + 2 * m)) & 3) * Hkv);
                    cp_async_arrive(&full[i_slot]);
                }
            } else {
                mbar_arrive(&full[i_slot]);
                if (scaled) mbar_arrive(&full[i_slot]);
            }
        }
        ++issued;
        if (++i_slot == nslots) i_slot = 0;
    };

    // ---- reading
    const int g = lane >> 2, c = lane & 3;
    // A lane's ldmatrix address of 16-byte chunks 2i, 2i + 1 of its row is
    // (row, chunk 0 or 1) with bit 5 + flipped by i: the swizzle only xors.
    // K (and 8-bit V) matrices are (tokens 0-7, chunk), (8-15, chunk),
    // (0-7, chunk + 1), (8-15, chunk + 1); bf16 V swaps the middle two.
    auto lane_at = [](int row, int ch) {
        if constexpr (C::kLine == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
        return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
    };
    const uint32_t k_at = ring + lane_at((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
    const uint32_t v_at =
        KIND == kWinBf16 ? ring + lane_at((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1) : k_at;
    constexpr int kPairs = C::kLine / 32;         // chunk pairs of one line
    // A slot holds one 16-token block after the other, panel by panel (with one
    // panel that is also what larger boxes write)
    constexpr int kPanel = 16 * C::kLine, kBlock = C::kPanels * kPanel;
    int slot = 0;
    uint32_t phase = 0;
    // False (for the whole warp) if the wait ran out.
    auto wait_full = [&]() {
        if (__all_sync(0xffffffffu, mbar_try_wait(&full[slot], phase))) return true;
        return __all_sync(0xffffffffu, wait_long(&full[slot], phase)) != 0;
    };
    auto refill = [&]() {  // the slot has been read
        __syncwarp();
        if (++slot == nslots) {
            slot = 0;
            phase ^= 1;
        }
        if (issued < loads) issue();
    };

    constexpr int kParts = 4 * NHB * C::kSteps / C::kHanded;  // of a warp's hand-over to another
    const int tiles = p1 - p0;
    int tile = 0;
    // Positions of a row block's rows, worked out where they are wanted (the
    // first tile and the edges): of the first and last row, and of row jr (rows
    // behind the last have its position).
    struct Rows {
        int first, last, skip;  // skip: rows of the first row's position before it
        __device__ __forceinline__ int at(const WinArgs& a, int jr) const {
            return MULTI ? min(first + a.grp_div(skip + jr), last) : last;
        }
    };
    auto rows_of = [&](int z) {
        const int v = z & kVMask, b = a.rb == 1 ? v : a.rb_div(v);
        const int row0 = a.rb == 1 ? 0 : (v - b * a.rb) * a.rbn, n = lens[b];
        if (!MULTI) return Rows{n - 1, n - 1, 0};
        const int i0 = a.grp_div(row0);
        return Rows{n - a.q_len + i0, n - a.q_len + a.grp_div(min(a.rows, row0 + a.rbn) - 1), row0 - i0 * a.grp};
    };
    uint32_t qb[NHB][C::kSteps][2];
    float o[NHB][C::kSteps][4];
    float m_ref[NHB][2], r_ref[NHB][2], l_part[NHB][2];

    for (; tile < tiles; ++tile) {
        // boxes are complete as many tiles ahead as copies run ahead of the
        // reader; the first time round the copies start before the second
        // chunk is located
        for (int step = tile == 0 ? 0 : completed < min(boxes, (tile + kMaxSlots / 2 + 1) * nb) ? 1 : 2; step < 2;
             ++step) {
            if (step == 1) {
                complete();
                if (tile == 0)
                    for (int s = 0; s < nslots && issued < loads; ++s) issue();
            }
            locate();
        }
        if ((tile & (kMeet - 1)) == kMeet - 1) named_bar_sync(1, 32 * NC);
        const int4 d = desc_s[(tile * nb) & (kDesc - 1)];
        const int t0 = d.x;

        if (d.z & kFirst) {
            const int v = d.z & kVMask, b = a.rb == 1 ? v : a.rb_div(v);
            const int row0 = a.rb == 1 ? 0 : (v - b * a.rb) * a.rbn;
            if (a.units > 0 && threadIdx.x == 0) {
                // every request's first and last unit, for the merge
                int2* u = a.ws_units + v;
                const int P = p0 + tile;
                if (P == cum[v]) u->x = blockIdx.x;
                if (cum[v + 1] <= p1) u->y = blockIdx.x;
            }
#pragma unroll
            for (int hb = 0; hb < NHB; ++hb) {
                // Q^T operand (row g): bf16, or f16 in the order of the codes' words
                const int R = row0 + hb * 8 + g;
                const int i = MULTI ? a.grp_div(R) : 0;
                const bool have = R < a.rows;
                const __nv_bfloat16* qr =
                    a.q + ((static_cast<long long>(b) * a.q_len + i) * a.Hq + kh * a.grp + (R - i * a.grp)) * D;
                if constexpr (KIND == kWinBf16) {
#pragma unroll
                    for (int ks = 0; ks < C::kSteps; ++ks) {
                        qb[hb][ks][0] = have ? __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * c)) : 0u;
                        qb[hb][ks][1] = have ? __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * c + 8)) : 0u;
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < C::kSteps; ++ks) {  // entries 16 ks + 4c .. + 3
                        const uint2 u = have ? __ldg(reinterpret_cast<const uint2*>(qr + ks * 16 + 4 * c))
                                             : make_uint2(0u, 0u);
                        qb[hb][ks][0] = q_f16(u.x);
                        qb[hb][ks][1] = q_f16(u.y);
                    }
                }
#pragma unroll
                for (int mb = 0; mb < C::kSteps; ++mb)
                    o[hb][mb][0] = o[hb][mb][1] = o[hb][mb][2] = o[hb][mb][3] = 0.f;
                m_ref[hb][0] = m_ref[hb][1] = r_ref[hb][0] = r_ref[hb][1] = kNone;
                l_part[hb][0] = l_part[hb][1] = 0.f;
            }
        }

        const bool any = d.z & (kBlocks * kAct);
        float x[MT][NHB][4];  // logits of token g (rows 2c, 2c + 1) and of token g + 8
        if (!wait_full()) break;
        if (any) {
            const uint32_t kb = k_at + slot * C::kSlot;
            // one chain of MMAs per (block, row group); two where there is one
            constexpr int kChains = MT * NHB == 1 ? 2 : 1;
            constexpr int kE = KIND == kWinBf16 ? 1 : 2;  // 16-wide steps of a chunk pair
            float st[kChains][MT][NHB][4];
            // blocks two by two; a pair without a visible key is passed over
#pragma unroll
            for (int m0 = 0; m0 < MT; m0 += 2) {
                const int m1 = m0 + 2 < MT ? m0 + 2 : MT;
                if (MT > 2 && !(d.z & (3 * kAct << m0))) {
#pragma unroll
                    for (int m = m0; m < m1; ++m)
#pragma unroll
                        for (int hb = 0; hb < NHB; ++hb)
                            st[0][m][hb][0] = st[0][m][hb][1] = st[0][m][hb][2] = st[0][m][hb][3] = 0.f;
                    continue;
                }
#pragma unroll
                for (int i = 0; i < C::kPanels * kPairs; ++i) {
                    uint32_t w[MT][4];
#pragma unroll
                    for (int m = m0; m < m1; ++m)
                        ldsm(w[m], (kb + (i / kPairs) * kPanel + m * kBlock) ^ ((i % kPairs) << 5));
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        const int ks = kE * i + e;
#pragma unroll
                        for (int m = m0; m < m1; ++m) {
                            uint32_t af[4] = {w[m][0], w[m][1], w[m][2], w[m][3]};
                            if constexpr (KIND != kWinBf16) {
                                const uint2 k0 = widen_adjacent<KIND>(w[m][2 * e]);
                                const uint2 k1 = widen_adjacent<KIND>(w[m][2 * e + 1]);
                                af[0] = k0.x;
                                af[1] = k1.x;
                                af[2] = k0.y;
                                af[3] = k1.y;
                            }
#pragma unroll
                            for (int hb = 0; hb < NHB; ++hb)
                                mma<KIND>(st[ks % kChains][m][hb], af, qb[hb][ks][0], qb[hb][ks][1], ks < kChains);
                        }
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float ksc = scaled ? a.sl2 * scale_s[slot * 4 + m] : a.sl2;
#pragma unroll
                for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[m][hb][e] =
                            (kChains == 1 ? st[0][m][hb][e] : st[0][m][hb][e] + st[kChains - 1][m][hb][e]) * ksc;
            }
        }
        refill();
        if (!wait_full()) break;
        if (any) {
            float lvs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) lvs[m] = scaled ? __log2f(scale_s[slot * 4 + m]) : 0.f;
            if (d.z & (kBlocks * kEdge)) {
                const Rows rows = rows_of(d.z);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (!(d.z & (kEdge << m))) continue;
                    const bool act = d.z & (kAct << m);
                    const int t = t0 + 16 * m;
                    if (!act) lvs[m] = 0.f;
#pragma unroll
                    for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {  // mask key by key
                            const int key = t + g + (e >> 1) * 8, p = rows.at(a, hb * 8 + 2 * c + (e & 1));
                            if (!act || !(key <= p && (key < a.sinks || key > p - a.window)))
                                x[m][hb][e] = -INFINITY;
                        }
                    if (MULTI && KIND != kWinBf16 && !(lvs[m] < INFINITY)) {
                        // an Inf or NaN scale, for the rows that see a key of
                        // it alone: their sums become NaN by way of the reference
#pragma unroll
                        for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (fmaxf(x[m][hb][e], x[m][hb][2 + e]) > -INFINITY) r_ref[hb][e] = NAN;
                        lvs[m] = 0.f;
                    }
                    if (KIND != kWinInt8) {
                        // V rows that no row sees become zeros: whatever bytes
                        // they hold (int8 codes are finite anyway)
                        const int r = lane >> 1, key = t + r;  // two lanes a row
                        if (!(act && key <= rows.last && (key < a.sinks || key > rows.first - a.window))) {
                            const uint32_t row = ring + slot * C::kSlot + m * kBlock + r * C::kLine + (lane & 1) * (C::kLine / 2);
#pragma unroll
                            for (int q = 0; q < C::kPanels; ++q)
#pragma unroll
                                for (int b16 = 0; b16 < C::kLine / 2; b16 += 16) st_shared_zero16(row + q * kPanel + b16);
                        }
                    }
                }
                if (KIND != kWinInt8) {
                    fence_proxy_async_smem();  // before the slot's next copy
                    __syncwarp();
                }
            }
            // the largest excess over a reference, in base-2 exponents
            float over = -INFINITY;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mx = fmaxf(x[m][hb][e], x[m][hb][2 + e]);
                        over = fmaxf(over, mx - m_ref[hb][e]);
                        if (KIND != kWinBf16) over = fmaxf(over, mx + (lvs[m] - r_ref[hb][e]));
                    }
            if (__any_sync(0xffffffffu, over > 8.f)) {
#pragma unroll
                for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = -INFINITY, mr = -INFINITY;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const float y = fmaxf(x[m][hb][e], x[m][hb][2 + e]);
                            mx = fmaxf(mx, y);
                            mr = fmaxf(mr, y + lvs[m]);
                        }
#pragma unroll
                        for (int s = 4; s <= 16; s <<= 1) {
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                            if (KIND != kWinBf16) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, s));
                        }
                        float f = 1.f;
                        if (mx > m_ref[hb][e] + 8.f) {
                            f = ex2(m_ref[hb][e] - mx);
                            l_part[hb][e] *= f;
                            m_ref[hb][e] = mx;
                        }
                        if (KIND != kWinBf16) {
                            f = 1.f;
                            if (mr > r_ref[hb][e] + 8.f) {
                                f = ex2(r_ref[hb][e] - mr);
                                r_ref[hb][e] = mr;
                            }
                        }
#pragma unroll
                        for (int mb = 0; mb < C::kSteps; ++mb) {
                            o[hb][mb][e] *= f;
                            o[hb][mb][2 + e] *= f;
                        }
                    }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (MT > 2 && !(d.z & (3 * kAct << (m & ~1)))) continue;
                const int t = t0 + 16 * m;
                // the sums take the fp32 probabilities; P.V takes them rounded
                uint32_t pb[NHB][2];
#pragma unroll
                for (int hb = 0; hb < NHB; ++hb) {
                    const float e0 = ex2(x[m][hb][0] - m_ref[hb][0]), e1 = ex2(x[m][hb][1] - m_ref[hb][1]);
                    const float e2 = ex2(x[m][hb][2] - m_ref[hb][0]), e3 = ex2(x[m][hb][3] - m_ref[hb][1]);
                    l_part[hb][0] += e0 + e2;
                    l_part[hb][1] += e1 + e3;
                    if (KIND != kWinBf16) {
                        const float d0 = lvs[m] - r_ref[hb][0], d1 = lvs[m] - r_ref[hb][1];
                        pb[hb][0] = movmatrix_t(p_pair<KIND>(ex2(x[m][hb][0] + d0), ex2(x[m][hb][1] + d1)));
                        pb[hb][1] = movmatrix_t(p_pair<KIND>(ex2(x[m][hb][2] + d0), ex2(x[m][hb][3] + d1)));
                    } else {
                        pb[hb][0] = movmatrix_t(p_pair<KIND>(e0, e1));
                        pb[hb][1] = movmatrix_t(p_pair<KIND>(e2, e3));
                    }
                }
                const uint32_t vb_at = v_at + slot * C::kSlot + m * kBlock;
                // operand A of head dims 16 mb ..: rows g and g + 8
                auto load_v = [&](int mb2, uint32_t (&av)[2][4], bool masked, uint2 k) {  // blocks 2 mb2, 2 mb2 + 1
                    if constexpr (KIND == kWinBf16) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = 2 * mb2 + e;
                            ldsm_t(av[e], (vb_at + (i / kPairs) * kPanel) ^ ((i % kPairs) << 5));
                            if (masked) {
                                av[e][0] &= k.x;
                                av[e][1] &= k.x;
                                av[e][2] &= k.y;
                                av[e][3] &= k.y;
                            }
                        }
                    } else {
                        uint32_t w[4];
                        ldsm_t(w, vb_at ^ (mb2 << 5));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (masked) {
                                w[2 * e] &= k.x;
                                w[2 * e + 1] &= k.y;
                            }
                            const uint2 lo2 = widen_strided<KIND>(w[2 * e]), hi2 = widen_strided<KIND>(w[2 * e + 1]);
                            av[e][0] = lo2.x;
                            av[e][1] = lo2.y;
                            av[e][2] = hi2.x;
                            av[e][3] = hi2.y;
                        }
                    }
                };
                bool apart = false;
                if (MULTI && KIND != kWinInt8 && (d.z & (kEdge << m))) {
                    // some key is seen by some rows only: is any V value Inf or NaN?
#pragma unroll
                    for (int i = 0; i < C::kPanels * kPairs; ++i) {
                        uint32_t w[4];
                        ldsm_t(w, (k_at + slot * C::kSlot + m * kBlock + (i / kPairs) * kPanel) ^
                                      ((i % kPairs) << 5));
                        apart |= non_finite<KIND>(w[0]) || non_finite<KIND>(w[1]) || non_finite<KIND>(w[2]) ||
                                 non_finite<KIND>(w[3]);
                    }
                    apart = __any_sync(0xffffffffu, apart);
                }
                if (!MULTI || !apart) {
#pragma unroll
                    for (int mb2 = 0; mb2 < C::kSteps / 2; ++mb2) {
                        uint32_t av[2][4];
                        load_v(mb2, av, false, make_uint2(0u, 0u));
#pragma unroll
                        for (int hb = 0; hb < NHB; ++hb) {
                            mma<KIND>(o[hb][2 * mb2], av[0], pb[hb][0], pb[hb][1]);
                            mma<KIND>(o[hb][2 * mb2 + 1], av[1], pb[hb][0], pb[hb][1]);
                        }
                    }
                } else {
                    const Rows rows = rows_of(d.z);
                    for (int p = rows.first; p <= rows.last; ++p) {  // one query position at a time
                        auto seen = [&](int key) { return key <= p && (key < a.sinks || key > p - a.window); };
                        const int key = t + 2 * c;  // V words hold tokens 2c, 2c + 1 (and + 8)
                        const uint2 k = make_uint2(
                            (seen(key) ? 0xffffu : 0u) | (seen(key + 1) ? 0xffff0000u : 0u),
                            (seen(key + 8) ? 0xffffu : 0u) | (seen(key + 9) ? 0xffff0000u : 0u));
#pragma unroll
                        for (int mb2 = 0; mb2 < C::kSteps / 2; ++mb2) {
                            uint32_t av[2][4];
                            load_v(mb2, av, true, k);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int hb = 0; hb < NHB; ++hb) {
                                    float s[4];
                                    mma<KIND>(s, av[e], pb[hb][0], pb[hb][1], true);
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        if (rows.at(a, hb * 8 + 2 * c + (y & 1)) == p)
                                            o[hb][2 * mb2 + e][y] += s[y];
                                }
                        }
                    }
                }
            }
        }
        refill();
        if (!(d.z & kLast)) continue;

        // ---- the rows' sums over the warp's lanes, then over the warps of
        // the head; references become -inf where there is none
#pragma unroll
        for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_part[hb][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                l_part[hb][e] = l;
                if (KIND == kWinBf16) r_ref[hb][e] = m_ref[hb][e];
                if (m_ref[hb][e] == kNone) m_ref[hb][e] = -INFINITY;
                if (r_ref[hb][e] == kNone) r_ref[hb][e] = -INFINITY;
            }
        if (TS > 1) {
            for (int half = TS / 2; half >= 1; half >>= 1) {
                // warp sub + half hands its state to warp sub
                float* buf = reinterpret_cast<float*>(smem + lay.exch) +
                             ((sub & (half - 1)) * Hkv + kh) * (C::kExch / 4) + lane;
                float* tail = buf + C::kHanded * 32;
                const bool gives = sub >= half && sub < 2 * half, takes = sub < half;
                float f0[NHB][2], f1[NHB][2];
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    if (gives) {
#pragma unroll
                        for (int y = 0; y < C::kHanded; ++y) {
                            const int i = part * C::kHanded + y;
                            buf[y * 32] = o[i / (4 * C::kSteps)][i / 4 % C::kSteps][i % 4];
                        }
                        if (part == 0)
#pragma unroll
                            for (int y = 0; y < 2 * NHB; ++y) {
                                tail[y * 96] = m_ref[y / 2][y % 2];
                                tail[y * 96 + 32] = r_ref[y / 2][y % 2];
                                tail[y * 96 + 64] = l_part[y / 2][y % 2];
                            }
                    }
                    named_bar_sync(1, 32 * NC);
                    if (takes) {
                        if (part == 0)
#pragma unroll
                            for (int y = 0; y < 2 * NHB; ++y) {
                                const int h = y / 2, e = y % 2;
                                const float m1 = tail[y * 96], r1 = tail[y * 96 + 32], l1 = tail[y * 96 + 64];
                                const float m = fmaxf(m_ref[h][e], m1), r = fmaxf(r_ref[h][e], r1);
                                const float mu = m == -INFINITY ? 0.f : m, ru = r == -INFINITY ? 0.f : r;
                                l_part[h][e] = l_part[h][e] * ex2(m_ref[h][e] - mu) + l1 * ex2(m1 - mu);
                                f0[h][e] = ex2(r_ref[h][e] - ru);
                                f1[h][e] = ex2(r1 - ru);
                                m_ref[h][e] = m;
                                r_ref[h][e] = r;
                            }
#pragma unroll
                        for (int y = 0; y < C::kHanded; ++y) {
                            const int i = part * C::kHanded + y, hb = i / (4 * C::kSteps);
                            float& x = o[hb][i / 4 % C::kSteps][i % 4];
                            x = x * f0[hb][i & 1] + buf[y * 32] * f1[hb][i & 1];
                        }
                    }
                    named_bar_sync(1, 32 * NC);
                }
            }
            if (sub > 0) continue;
        }

        // ---- epilogue: rows hb * 8 + 2c + e; head dims by kind (see the top)
        const int v = d.z & kVMask, b = a.rb == 1 ? v : a.rb_div(v);
        const int row0 = a.rb == 1 ? 0 : (v - b * a.rb) * a.rbn;
#pragma unroll
        for (int hb = 0; hb < NHB; ++hb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int jr = hb * 8 + 2 * c + e, R = row0 + jr;
                if (jr >= a.rbn || R >= a.rows) continue;
                const float l = l_part[hb][e];
                // l == 0: no visible key (a NaN sum goes through to the output)
                float f = 0.f;
                if (l != 0.f)
                    f = a.out_scale * (r_ref[hb][e] == -INFINITY ? 0.f : ex2(r_ref[hb][e] - m_ref[hb][e])) / l;
                const float lse = l != 0.f ? (m_ref[hb][e] + log2f(l)) * kLn2 : -INFINITY;
                if (d.z & kWhole) {
                    const int i = MULTI ? a.grp_div(R) : 0;
                    const long long orow =
                        (static_cast<long long>(b) * a.q_len + i) * a.Hq + kh * a.grp + (R - i * a.grp);
                    __nv_bfloat16* op = a.out + orow * D;
#pragma unroll
                    for (int mb = 0; mb < C::kSteps; ++mb) {
                        if constexpr (KIND == kWinBf16) {
                            op[mb * 16 + g] = __float2bfloat16_rn(o[hb][mb][e] * f);
                            op[mb * 16 + g + 8] = __float2bfloat16_rn(o[hb][mb][2 + e] * f);
                        } else {
                            *reinterpret_cast<uint32_t*>(op + mb * 16 + 2 * g) =
                                pack_bf16x2(o[hb][mb][e] * f, o[hb][mb][2 + e] * f);
                        }
                    }
                    if (a.lse && g == 0) a.lse[orow] = lse;
                } else {
                    const long long prow =
                        (static_cast<long long>(static_cast<int>(blockIdx.x) + v) * Hkv + kh) * a.rbn + jr;
                    float* op = a.ws_o + prow * D;
#pragma unroll
                    for (int mb = 0; mb < C::kSteps; ++mb) {
                        if constexpr (KIND == kWinBf16) {
                            op[mb * 16 + g] = o[hb][mb][e] * f;
                            op[mb * 16 + g + 8] = o[hb][mb][2 + e] * f;
                        } else {
                            *reinterpret_cast<float2*>(op + mb * 16 + 2 * g) =
                                make_float2(o[hb][mb][e] * f, o[hb][mb][2 + e] * f);
                        }
                    }
                    if (g == 0) a.ws_lse[prow] = lse;
                }
            }
    }
    if (tile < tiles) {
        // A wait ran out: report it, meet the other warps wherever they
        // expect it, write nothing more, and let the copies in flight land
        // (bounded like every wait; a landed fill's phase answers at once).
        report(a.status, MQA_ERR_DEVICE_TIMEOUT);
        for (int t = tile; t < tiles; ++t) {
            if (t > tile && (t & (kMeet - 1)) == kMeet - 1) named_bar_sync(1, 32 * NC);
            if (completed < min(boxes, (t + kMaxSlots / 2 + 1) * nb)) {
                complete();
                locate();
            }
            if (desc_s[(t * nb) & (kDesc - 1)].z & kLast)
                for (int half = TS / 2; half >= 1; half >>= 1)
                    for (int part = 0; part < 2 * kParts; ++part) named_bar_sync(1, 32 * NC);
        }
        for (int s = 0; s < nslots && s < issued; ++s) {
            const int fills = (issued - s + nslots - 1) / nslots;
            if (!mbar_wait(&full[s], (fills - 1) & 1)) break;
        }
    }
}

// Lets `kern` (one of the two of this instance) use all of a block's shared
// memory, once per device.
template <int D, int KIND, int NHB>
cudaError_t allow_smem(const void* kern, bool multi) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[2][kDevices];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (known && done[multi][dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (known && e == cudaSuccess) done[multi][dev].store(true, std::memory_order_relaxed);
    return e;
}

template <int D, int KIND, int NHB>
cudaError_t launch(WinArgs a, int grid, cudaStream_t stream) {
    const int vb = a.batch * a.rb;
    const int limit = 228 * 1024 / (a.alone ? 1 : win_ctas_per_sm(NHB, D)) - 1024;  // a block's share of an SM's
    int ns = kMaxSlots;
    while (ns > 2 && layout<D, KIND, NHB>(a.Hkv, a.ts, ns, vb, a.batch).total > limit) --ns;
    a.nslots = ns;
    const int bytes = layout<D, KIND, NHB>(a.Hkv, a.ts, ns, vb, a.batch).total;
    // (more than 16 rows of a KV head are several positions')
    auto kern = NHB > 2 || a.q_len > 1 ? gqa_win_kernel<D, KIND, NHB, true>
                                       : gqa_win_kernel<D, KIND, NHB <= 2 ? NHB : 1, false>;
    if (cudaError_t e = allow_smem<D, KIND, NHB>(reinterpret_cast<const void*>(kern), a.q_len > 1); e != cudaSuccess) return e;
    return launch_with_pdl(kern, dim3(grid), dim3(32 * a.Hkv * a.ts), bytes, stream, a);
}

template <int D, int KIND>
cudaError_t dispatch_rows(const WinArgs& a, int grid, cudaStream_t stream) {
    switch (win_row_groups(a.rbn)) {
        case 1: return launch<D, KIND, 1>(a, grid, stream);
        case 2: return launch<D, KIND, 2>(a, grid, stream);
        default: return launch<D, KIND, 3>(a, grid, stream);
    }
}

template <int KIND>
cudaError_t dispatch(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    return D == 128 ? dispatch_rows<128, KIND>(a, grid, stream) : dispatch_rows<64, KIND>(a, grid, stream);
}

}  // namespace win
}  // namespace mqa

// Appending new tokens to a paged cache, the rotary position applied on the way.
//
// Token t of the ragged batch belongs to the request b with query_start[b] <=
// t < query_start[b + 1] and sits at position p = seq_lens[b] -
// (query_start[b + 1] - t).  A pair (x, y) of a query or key row becomes
// (x c - y s, y c + x s) with c, s the cosine and sine of row p of the table;
// pairs are halves apart or side by side.  The row goes to slot p % page of
// physical block block_table[b][p / page], in the cache's format.
//
// Bound by the bytes of the new rows (read once, written once) and, for one
// decode step, by the chain of dependent loads length -> block id / angle ->
// store.  So a lane owns both halves of its 8 pairs (two 16-byte loads, two
// stores, no exchange between lanes; a row may be rotated in place), the loads
// of a warp's rows are issued before the chain, and the angles are read once
// for all heads of a token.  fp32 arithmetic, one rounding at the store.
//
// Block-scaled formats: one warp owns one (block of tokens, plane, head).  It
// takes the largest magnitude of the new values, s = max(s_old, amax / Q) (s_old
// only where the block already held tokens), rescales the codes it held by
// s_old / s if the scale grew, and stores the new codes x / s.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "api_common.cuh"
#include "append.cuh"

namespace mqa {
namespace {

constexpr int kWarps = 4;
// Thread blocks per SM that the registers are limited for.  5 / 6 / 8: 6 prompts
// (8700 tokens, 32/8 heads x 128) bf16 39.9 / 37.7 / 40.6 us, e4m3 blocks 37.6 /
// 37.4 / 39.5; 1024 runs of 64 tokens (8/8 x 128, held codes) 163 / 157 / 156; 256
// runs of one token, bf16 3.1 / 3.1 / 3.7.  At 6 the block formats spill 52 bytes
// a thread, which costs them nothing that 5, without spills, would give back.
constexpr int kCtas = 6;
constexpr float kE4m3Max = 448.f, kInt8Max = 127.f, kInt4Max = 7.f;
constexpr float kTinyScale = 1.1754943508222875e-38f;  // 2^-126: scales are zero or normal

// The request that token t belongs to, with its entries; false for padding.
// query_start ascends: a warp narrows the candidates to 32 by samples, then
// reads those with their lengths, so that a batch of up to 32 (1024) requests
// costs one (two) dependent loads.
struct Owner {
    int b, q0, q1, len;
};
__device__ __forceinline__ bool find_owner(const AppendBatch& a, int t, int lane, Owner& o) {
    int lo = 0, n = a.batch;
    while (n > 32) {
        const int step = (n + 31) / 32, at = lane * step;
        const int m = __popc(__ballot_sync(0xffffffffu, at < n && __ldg(a.query_start + lo + at) <= t));
        if (m == 0) return false;
        lo += (m - 1) * step;
        n = min(step, n - (m - 1) * step);
    }
    int q0 = 0, q1 = 0, len = 0;
    if (lane < n) {
        q0 = __ldg(a.query_start + lo + lane);
        q1 = __ldg(a.query_start + lo + lane + 1);
        len = __ldg(a.seq_lens + lo + lane);
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, lane < n && q0 <= t && t < q1);
    if (hit == 0) return false;
    const int s = __ffs(hit) - 1;
    o.b = lo + s;
    o.q0 = __shfl_sync(0xffffffffu, q0, s);
    o.q1 = __shfl_sync(0xffffffffu, q1, s);
    o.len = __shfl_sync(0xffffffffu, len, s);
    return true;
}

// Position of token t of request o, or -1 (reported) where the request's
// length does not hold its new tokens or the position has no angle or page.
__device__ __forceinline__ int position(const AppendBatch& a, const Owner& o, int t) {
    const long long p = static_cast<long long>(o.len) - o.q1 + t;
    if (o.q0 < 0 || o.q1 > a.tokens || o.len < static_cast<long long>(o.q1) - o.q0 || p >= a.max_position ||
        p >= static_cast<long long>(a.max_blocks) * a.page) {
        report(a.status, MQA_ERR_DEVICE_CHECK);
        return -1;
    }
    return static_cast<int>(p);
}

__device__ __forceinline__ int block_id(const AppendBatch& a, int b, int p) {
    const int id = __ldg(a.block_table + static_cast<long long>(b) * a.max_blocks + p / a.page);
    if (id < 0 || id >= a.num_blocks) {
        report(a.status, MQA_ERR_DEVICE_CHECK);
        return -1;
    }
    return id;
}

// The two 8-element chunks (first columns c0, c1) that lane l of a row owns,
// and whether they are rotated: pairs 8l .. 8l + 7 of the rotary part, or 16
// columns behind it.
struct Chunks {
    int c0, c1;
    bool rot;
};
__device__ __forceinline__ Chunks chunks_of(int l, int rotary, bool interleaved) {
    const int lr = rotary / 16;
    if (l >= lr || interleaved) return {16 * l, 16 * l + 8, l < lr};
    return {8 * l, 8 * l + rotary / 2, true};
}

struct Angles {
    float c[8], s[8];
};
__device__ __forceinline__ void load_angles(Angles& an, const AppendBatch& a, int p, int l) {
    const float* row = a.cos_sin + static_cast<long long>(p) * a.rotary + 8 * l;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<float4*>(an.c + 4 * i) = __ldg(reinterpret_cast<const float4*>(row) + i);
        *reinterpret_cast<float4*>(an.s + 4 * i) = __ldg(reinterpret_cast<const float4*>(row + a.rotary / 2) + i);
    }
}

__device__ __forceinline__ void unpack8(float (&y)[8], uint4 v) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(u[i] << 16);
        y[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
}

// The 16 values of a lane's chunks, rotated.
__device__ __forceinline__ void rotate(float (&y0)[8], float (&y1)[8], const Angles& an, bool interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (interleaved) {
            float& x = i < 4 ? y0[(2 * i) & 7] : y1[(2 * i) & 7];
            float& y = i < 4 ? y0[(2 * i + 1) & 7] : y1[(2 * i + 1) & 7];
            const float a = x * an.c[i] - y * an.s[i], b = y * an.c[i] + x * an.s[i];
            x = a;
            y = b;
        } else {
            const float a = y0[i] * an.c[i] - y1[i] * an.s[i], b = y1[i] * an.c[i] + y0[i] * an.s[i];
            y0[i] = a;
            y1[i] = b;
        }
    }
}

__device__ __forceinline__ int int_code(float x, float top) { return __float2int_rn(fminf(fmaxf(x, -top), top)); }
// Four 8-bit codes, lowest first; INT8 selects the format.  (int8: |x| is at
// most 127 and a rounding, so that saturation to -128 does not come up.)
template <bool INT8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint32_t r;
    if constexpr (INT8) {
        asm("{\n\t.reg .b32 t;\n\tcvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\t"
            "cvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}"
            : "=r"(r)
            : "r"(__float2int_rn(a)), "r"(__float2int_rn(b)), "r"(__float2int_rn(c)), "r"(__float2int_rn(d)));
    } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    }
    return r;
}
// The eight codes of y / s, given inv = 1 / s (0 where s = 0: zeros).  The
// product is within 2^-23 of the quotient, relative: another code only where
// the quotient is that near the border between two.
template <bool INT8>
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
    if (inv == 0.f) return make_uint2(0u, 0u);  // (a product could be -0)
    return make_uint2(codes4<INT8>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                      codes4<INT8>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}
__device__ __forceinline__ float inverse(float s) { return s == 0.f ? 0.f : 1.f / s; }

__device__ __forceinline__ float amax16(const float (&y0)[8], const float (&y1)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(y0[i]), fabsf(y1[i])));
    return m;
}

// Bytes of one (token, head) row of a GQA cache.
template <int D, int FMT>
__device__ __host__ constexpr int row_bytes() {
    return FMT == MQA_KV_BF16                  ? 2 * D
           : FMT == MQA_KV_INT4_PER_TOKEN_HEAD ? D / 2 + 4
           : (FMT == MQA_KV_FP8_E4M3_PER_TOKEN_HEAD || FMT == MQA_KV_INT8_PER_TOKEN_HEAD) ? D + 4
                                                                                          : D;
}

// Stores a lane's 16 values of one cache row (not the block-scaled formats);
// D / 16 lanes hold the row.  Per-token-head formats: all lanes of the warp
// call it.
template <int D, int FMT>
__device__ __forceinline__ void store_row(uint8_t* row, bool store, const float (&y0)[8], const float (&y1)[8],
                                          int c0, int c1, int l, float tensor_inv) {
    if constexpr (FMT == MQA_KV_BF16) {
        if (!store) return;
        *reinterpret_cast<uint4*>(row + 2 * c0) = pack8(y0);
        *reinterpret_cast<uint4*>(row + 2 * c1) = pack8(y1);
    } else if constexpr (FMT == MQA_KV_FP8_E4M3) {
        if (!store) return;
        *reinterpret_cast<uint2*>(row + c0) = codes8<false>(y0, tensor_inv);
        *reinterpret_cast<uint2*>(row + c1) = codes8<false>(y1, tensor_inv);
    } else {
        constexpr float top = FMT == MQA_KV_FP8_E4M3_PER_TOKEN_HEAD ? kE4m3Max
                              : FMT == MQA_KV_INT8_PER_TOKEN_HEAD   ? kInt8Max
                                                                    : kInt4Max;
        float m = amax16(y0, y1);
#pragma unroll
        for (int o = D / 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = m / top;
        if (s < kTinyScale) s = 0.f;
        if (!store) return;
        const float inv = inverse(s);
        if constexpr (FMT == MQA_KV_INT4_PER_TOKEN_HEAD) {
            auto word = [&](const float (&y)[8]) {
                uint32_t w = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w |= (static_cast<uint32_t>(int_code(y[i] * inv, kInt4Max)) & 0xfu) << (4 * i);
                return w;
            };
            *reinterpret_cast<uint32_t*>(row + c0 / 2) = word(y0);
            *reinterpret_cast<uint32_t*>(row + c1 / 2) = word(y1);
            if (l == 0) *reinterpret_cast<float*>(row + D / 2) = s;
        } else {
            constexpr bool int8 = FMT == MQA_KV_INT8_PER_TOKEN_HEAD;
            const uint2 a = codes8<int8>(y0, inv), b = codes8<int8>(y1, inv);
            reinterpret_cast<uint32_t*>(row + c0)[0] = a.x;  // rows of D + 4 bytes: 4-byte alignment
            reinterpret_cast<uint32_t*>(row + c0)[1] = a.y;
            reinterpret_cast<uint32_t*>(row + c1)[0] = b.x;
            reinterpret_cast<uint32_t*>(row + c1)[1] = b.y;
            if (l == 0) *reinterpret_cast<float*>(row + D) = s;
        }
    }
}

// Rows of a token that one warp takes: kIter passes of 32 / (D / 16) rows.
constexpr int kIter = 4;

template <int D>
__host__ __device__ constexpr int rows_per_warp() {
    return kIter * (32 / (D / 16));
}

template <int FMT>
__host__ __device__ constexpr bool block_format() {
    return FMT == MQA_KV_FP8_E4M3_BLOCK || FMT == MQA_KV_INT8_BLOCK;
}

// One token's rows [r0, r0 + rows_per_warp): query rows, then (unless the
// format is block-scaled) key and value rows.
template <int D, int FMT>
__device__ __forceinline__ void append_rows(const GqaAppendArgs& a, int t, int r0, int lane) {
    constexpr int LPR = D / 16, RPI = 32 / LPR;
    constexpr bool BLOCK = block_format<FMT>();
    const int l = lane % LPR;
    const Chunks ch = chunks_of(l, a.t.rotary, a.t.interleaved);
    const int rows = a.Hq + (BLOCK ? 0 : 2 * a.Hkv);
    uint4 x0[kIter], x1[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int r = r0 + it * RPI + lane / LPR;
        x0[it] = x1[it] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= rows) continue;
        const __nv_bfloat16* src = r < a.Hq           ? a.q + t * a.q_stride + r * D
                                   : r < a.Hq + a.Hkv ? a.k + t * a.k_stride + (r - a.Hq) * D
                                                      : a.v + t * a.v_stride + (r - a.Hq - a.Hkv) * D;
        x0[it] = *reinterpret_cast<const uint4*>(src + ch.c0);
        x1[it] = *reinterpret_cast<const uint4*>(src + ch.c1);
    }
    Owner own;
    if (!find_owner(a.t, t, lane, own)) return;  // padding: no request's token
    const int p = position(a.t, own, t);
    if (p < 0) return;
    Angles an;
    if (ch.rot) load_angles(an, a.t, p, l);
    const int id = BLOCK ? -1 : block_id(a.t, own.b, p);
    uint8_t* cell = a.cache + (static_cast<long long>(id) * 2 * a.t.page + p % a.t.page) * a.Hkv * row_bytes<D, FMT>();
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        if (r0 + it * RPI >= rows) break;  // warp-uniform
        const int r = r0 + it * RPI + lane / LPR;
        float y0[8], y1[8];
        unpack8(y0, x0[it]);
        unpack8(y1, x1[it]);
        if (ch.rot && r < a.Hq + a.Hkv) rotate(y0, y1, an, a.t.interleaved);
        if (r < a.Hq) {
            __nv_bfloat16* dst = a.q_out + t * a.qo_stride + r * D;
            *reinterpret_cast<uint4*>(dst + ch.c0) = pack8(y0);
            *reinterpret_cast<uint4*>(dst + ch.c1) = pack8(y1);
        }
        if constexpr (!BLOCK) {
            const int h = r - a.Hq;  // key rows, then value rows
            const bool v = h >= a.Hkv;
            uint8_t* row = cell + (static_cast<long long>(v) * a.t.page * a.Hkv + (v ? h - a.Hkv : h)) * row_bytes<D, FMT>();
            store_row<D, FMT>(row, h >= 0 && r < rows && id >= 0, y0, y1, ch.c0, ch.c1, l,
                              FMT == MQA_KV_FP8_E4M3 ? 1.f / (v ? a.v_scale : a.k_scale) : 0.f);
        }
    }
}

// Four 8-bit codes rescaled: round(code * ratio).
template <bool INT8>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (INT8) {
            f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
        } else {
            const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(w >> (8 * i)), __NV_E4M3);
            f[i] = __half2float(*reinterpret_cast<const __half*>(&h));
        }
        f[i] *= ratio;
    }
    return codes4<INT8>(f[0], f[1], f[2], f[3]);
}

// A request's share of a block of tokens: its new positions [pa, pe) of the
// block starting at position `first`, the first of them token t.
struct Share {
    int b, first, pa, pe, t;
};
__device__ __forceinline__ bool share_of(const AppendBatch& a, const Owner& o, int p0, int first, int G, Share& s) {
    const long long last = static_cast<long long>(first) + G;
    s.b = o.b;
    s.first = first;
    s.pa = max(p0, first);
    s.pe = static_cast<int>(last < o.len ? last : static_cast<long long>(o.len));
    s.t = o.q0 + s.pa - p0;
    if (s.pe > a.max_position || s.pe > static_cast<long long>(a.max_blocks) * a.page) {
        report(a.status, MQA_ERR_DEVICE_CHECK);
        return false;
    }
    return true;
}

// The share that starts with token t, if one does.
__device__ __forceinline__ bool share_at_token(const AppendBatch& a, int t, int G, int lane, Share& s) {
    Owner o;
    if (!find_owner(a, t, lane, o)) return false;
    const long long p0 = static_cast<long long>(o.len) - (static_cast<long long>(o.q1) - o.q0);
    if (o.q0 < 0 || o.q1 > a.tokens || p0 < 0) {
        if (t == o.q0) report(a.status, MQA_ERR_DEVICE_CHECK);
        return false;
    }
    const int p = static_cast<int>(p0) + (t - o.q0);
    if (t != o.q0 && p % G != 0) return false;
    return share_of(a, o, static_cast<int>(p0), p / G * G, G, s);
}

// Share number `task`: request b's shares are numbered from query_start[b] / G
// + 2 b on, which leaves room for the (n - 1) / G + 2 that its n tokens touch
// at most and ascends without a sum over the batch.  The request is found as in
// find_owner.
__device__ __forceinline__ bool share_by_number(const AppendBatch& a, long long task, int G, int lane, Share& s) {
    auto number = [&](int b) { return __ldg(a.query_start + b) / G + 2LL * b; };
    int lo = 0, n = a.batch;
    while (n > 32) {
        const int step = (n + 31) / 32, at = lane * step;
        const int m = __popc(__ballot_sync(0xffffffffu, at < n && number(lo + at) <= task));
        if (m == 0) return false;
        lo += (m - 1) * step;
        n = min(step, n - (m - 1) * step);
    }
    Owner o{lo + lane, 0, 0, 0};
    long long at = 0;
    if (lane < n) {
        o.q0 = __ldg(a.query_start + o.b);
        o.q1 = __ldg(a.query_start + o.b + 1);
        o.len = __ldg(a.seq_lens + o.b);
        at = o.q0 / G + 2LL * o.b;
    }
    const int m = __popc(__ballot_sync(0xffffffffu, lane < n && at <= task));
    if (m == 0) return false;
    o.b = __shfl_sync(0xffffffffu, o.b, m - 1);
    o.q0 = __shfl_sync(0xffffffffu, o.q0, m - 1);
    o.q1 = __shfl_sync(0xffffffffu, o.q1, m - 1);
    o.len = __shfl_sync(0xffffffffu, o.len, m - 1);
    if (o.q1 <= o.q0) return false;  // no new tokens
    if (o.q0 < 0 || o.q1 > a.tokens || o.len < static_cast<long long>(o.q1) - o.q0) {
        report(a.status, MQA_ERR_DEVICE_CHECK);
        return false;
    }
    const int p0 = o.len - (o.q1 - o.q0);
    const long long kth = task - __shfl_sync(0xffffffffu, at, m - 1);
    if (kth < 0 || kth > (o.len - 1) / G - p0 / G) return false;
    return share_of(a, o, p0, (p0 / G + static_cast<int>(kth)) * G, G, s);
}

// How a share is found: at the token that starts it, or by its number; and by how many warps of a thread block it is then done.
struct ShareMode {
    bool by_token;
    int warps;  // 1 or kWarps
};

// Block-scaled formats: one share, one plane and head, rows dealt to
// mode.warps warps (a warp alone, or a whole thread block).
template <int D, int FMT>
__device__ __forceinline__ void append_block(const GqaAppendArgs& a, long long task, ShareMode mode, int plane, int head,
                                             int lane, float* exchange) {
    constexpr int LPR = D / 16, RPI = 32 / LPR;
    constexpr bool INT8 = FMT == MQA_KV_INT8_BLOCK;
    constexpr float top = INT8 ? kInt8Max : kE4m3Max;
    const int G = a.scale_block;
    Share sh;
    if (!(mode.by_token ? share_at_token(a.t, static_cast<int>(task), G, lane, sh)
                   : share_by_number(a.t, task, G, lane, sh)))
        return;
    const int first = sh.first, pa = sh.pa, pe = sh.pe;
    const int had = pa - first, m = pe - pa;
    const int warp = mode.warps == 1 ? 0 : threadIdx.x >> 5;
    const int l = lane % LPR, rl = lane / LPR + warp * RPI, step = RPI * mode.warps;
    const Chunks ch = chunks_of(l, a.t.rotary, a.t.interleaved);
    const bool rot = plane == 0 && ch.rot;
    const long long stride = plane ? a.v_stride : a.k_stride;
    const __nv_bfloat16* src = (plane ? a.v : a.k) + sh.t * stride + head * D;
    // up to kKeep new rows per lane are read once and kept; the rest twice
    constexpr int kKeep = 4;
    uint4 x0[kKeep], x1[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = rl + k * step;
        x0[k] = x1[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i >= m) continue;
        x0[k] = *reinterpret_cast<const uint4*>(src + i * stride + ch.c0);
        x1[k] = *reinterpret_cast<const uint4*>(src + i * stride + ch.c1);
    }
    const int id = block_id(a.t, sh.b, first);
    if (id < 0) return;
    const int slot = first % a.t.page;
    float* sp = a.scales + ((static_cast<long long>(id) * 2 + plane) * (a.t.page / G) + slot / G) * a.Hkv + head;
    const float s_old = had > 0 ? *sp : 0.f;
    uint8_t* cell = a.cache + (((static_cast<long long>(id) * 2 + plane) * a.t.page + slot) * a.Hkv + head) * D;
    const long long row_step = static_cast<long long>(a.Hkv) * D;

    // values of new row i < m, given its chunks
    auto values = [&](int i, uint4 u0, uint4 u1, float (&y0)[8], float (&y1)[8]) {
        unpack8(y0, u0);
        unpack8(y1, u1);
        if (rot) {
            Angles an;
            load_angles(an, a.t, pa + i, l);
            rotate(y0, y1, an, a.t.interleaved);
        }
    };
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = rl + k * step;
        if (i >= m) continue;
        float y0[8], y1[8];
        values(i, x0[k], x1[k], y0, y1);
        amax = fmaxf(amax, amax16(y0, y1));
    }
#pragma unroll 2
    for (int i = rl + kKeep * step; i < m; i += step) {
        float y0[8], y1[8];
        values(i, *reinterpret_cast<const uint4*>(src + i * stride + ch.c0),
               *reinterpret_cast<const uint4*>(src + i * stride + ch.c1), y0, y1);
        amax = fmaxf(amax, amax16(y0, y1));
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (mode.warps > 1) {  // (every warp has read s_old by the time it meets the others)
        if (lane == 0) exchange[warp] = amax;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, exchange[w]);
    }
    float s_new = amax / top;
    if (s_new < kTinyScale) s_new = 0.f;
    s_new = fmaxf(s_new, s_old);
    if (s_new > s_old && had > 0) {  // the codes the block held, at the new scale
        const float ratio = s_old / s_new;
        for (int i = rl; i < had; i += step) {
            uint4* p = reinterpret_cast<uint4*>(cell + i * row_step + 16 * l);
            const uint4 w = *p;
            *p = make_uint4(rescale4<INT8>(w.x, ratio), rescale4<INT8>(w.y, ratio), rescale4<INT8>(w.z, ratio),
                            rescale4<INT8>(w.w, ratio));
        }
    }
    const float inv = inverse(s_new);
    auto store = [&](int i, const float (&y0)[8], const float (&y1)[8]) {
        uint8_t* row = cell + (had + i) * row_step;
        *reinterpret_cast<uint2*>(row + ch.c0) = codes8<INT8>(y0, inv);
        *reinterpret_cast<uint2*>(row + ch.c1) = codes8<INT8>(y1, inv);
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = rl + k * step;
        if (i >= m) continue;
        float y0[8], y1[8];
        values(i, x0[k], x1[k], y0, y1);
        store(i, y0, y1);
    }
#pragma unroll 2
    for (int i = rl + kKeep * step; i < m; i += step) {
        float y0[8], y1[8];
        values(i, *reinterpret_cast<const uint4*>(src + i * stride + ch.c0),
               *reinterpret_cast<const uint4*>(src + i * stride + ch.c1), y0, y1);
        store(i, y0, y1);
    }
    if (lane == 0 && warp == 0) *sp = s_new;
}

// Warp tasks: (block formats) blocks, which take longest, then rows of tokens.
template <int D, int FMT>
__global__ void __launch_bounds__(32 * kWarps, kCtas) gqa_append_kernel(const GqaAppendArgs a, const int groups,
                                                                 const long long row_tasks,
                                                                 const long long block_tasks, const ShareMode mode) {
    __shared__ float exchange[kWarps];
    const int lane = threadIdx.x & 31;
    long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (block_format<FMT>()) {
        // (whole thread blocks where several warps share a task)
        const long long k = mode.warps == 1 ? w : blockIdx.x;
        if (k < block_tasks) {
            const long long task = k / (2 * a.Hkv);
            const int ph = static_cast<int>(k - task * 2 * a.Hkv);
            append_block<D, FMT>(a, task, mode, ph / a.Hkv, ph % a.Hkv, lane, exchange);
            return;
        }
        w -= block_tasks * mode.warps;
    }
    if (w >= row_tasks) return;
    const int t = static_cast<int>(w / groups);
    append_rows<D, FMT>(a, t, static_cast<int>(w - static_cast<long long>(t) * groups) * rows_per_warp<D>(), lane);
}

// MLA: a token's 64-column pieces: R / 64 of kv_c, k_pe, then H of q_pe (4
// lanes a piece).
template <bool FP8>
__global__ void __launch_bounds__(32 * kWarps, kCtas) mla_append_kernel(const MlaAppendArgs a, const int groups,
                                                                 const long long row_tasks) {
    constexpr int D = 64, LPR = 4, RPI = 8;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (w >= row_tasks) return;
    const int t = static_cast<int>(w / groups);
    const int r0 = static_cast<int>(w - static_cast<long long>(t) * groups) * kIter * RPI;
    const int l = lane % LPR;
    const int nc = a.R / 64, pieces = nc + 1 + a.H;
    const Chunks ch = chunks_of(l, 64, a.t.interleaved);
    uint4 x0[kIter], x1[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int r = r0 + it * RPI + lane / LPR;
        x0[it] = x1[it] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= pieces) continue;
        const __nv_bfloat16* src = r < nc    ? a.kv_c + t * a.c_stride + r * 64
                                   : r == nc ? a.k_pe + t * a.p_stride
                                             : a.q_pe + t * a.q_stride + (r - nc - 1) * a.qh_stride;
        x0[it] = *reinterpret_cast<const uint4*>(src + ch.c0);
        x1[it] = *reinterpret_cast<const uint4*>(src + ch.c1);
    }
    Owner own;
    if (!find_owner(a.t, t, lane, own)) return;  // padding
    const int p = position(a.t, own, t);
    if (p < 0) return;
    Angles an;
    load_angles(an, a.t, p, l);
    const int id = r0 <= nc ? block_id(a.t, own.b, p) : -1;
    uint8_t* cell = a.cache + (static_cast<long long>(id) * a.t.page + p % a.t.page) * (a.R + 64) * (FP8 ? 1 : 2);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int r = r0 + it * RPI + lane / LPR;
        if (r >= pieces) continue;
        float y0[8], y1[8];
        unpack8(y0, x0[it]);
        unpack8(y1, x1[it]);
        if (r >= nc) rotate(y0, y1, an, a.t.interleaved);
        if (r > nc) {
            __nv_bfloat16* dst = a.q_out + t * a.qo_stride + (r - nc - 1) * a.qoh_stride;
            *reinterpret_cast<uint4*>(dst + ch.c0) = pack8(y0);
            *reinterpret_cast<uint4*>(dst + ch.c1) = pack8(y1);
        } else {
            store_row<D, FP8 ? MQA_KV_FP8_E4M3 : MQA_KV_BF16>(cell + r * 64 * (FP8 ? 1 : 2), id >= 0, y0, y1, ch.c0,
                                                              ch.c1, l, FP8 ? 1.f / a.k_scale : 0.f);
        }
    }
}

template <int D, int FMT>
cudaError_t launch(const GqaAppendArgs& a, cudaStream_t stream) {
    constexpr bool BLOCK = block_format<FMT>();
    const int rows = a.Hq + (BLOCK ? 0 : 2 * a.Hkv);
    const int groups = (rows + rows_per_warp<D>() - 1) / rows_per_warp<D>();
    const long long row_tasks = static_cast<long long>(a.t.tokens) * groups;
    long long block_tasks = 0;
    ShareMode mode{false, 1};
    if (BLOCK) {
        // One task per plane, head and share of a block, or per token where
        // that is less (a request with n new tokens touches at most n blocks,
        // and at most (n - 1) / G + 2).
        const long long T = a.t.tokens, bound = T / a.scale_block + 2LL * a.t.batch;
        mode.by_token = T <= bound;
        // Shares of some length go to four warps while there are not enough of
        // them to fill the device's: a warp alone waits for its rows' loads in
        // turn, twice.  Blocks of 64 tokens, 8 heads x 128, int8, one warp / four:
        // 32 runs of 64 (100) new tokens 17 (20) / 13 (13) us, 128 runs of 64
        // 25 / 27 us, 1024 runs 137 / 195 us.
        const long long warps = static_cast<long long>(api_sm_count()) * kCtas * kWarps;
        mode.warps = T > 8 * bound && bound * 2 * a.Hkv <= warps ? kWarps : 1;
        block_tasks = (mode.by_token ? T : bound) * 2 * a.Hkv;
    }
    const long long grid = (row_tasks + block_tasks * mode.warps + kWarps - 1) / kWarps;
    return launch_with_pdl(gqa_append_kernel<D, FMT>, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), 0, stream,
                           a, groups > 0 ? groups : 1, row_tasks, block_tasks, mode);
}

template <int D>
cudaError_t dispatch(const GqaAppendArgs& a, int kv_dtype, cudaStream_t stream) {
    switch (kv_dtype) {
        case MQA_KV_BF16: return launch<D, MQA_KV_BF16>(a, stream);
        case MQA_KV_FP8_E4M3: return launch<D, MQA_KV_FP8_E4M3>(a, stream);
        case MQA_KV_FP8_E4M3_PER_TOKEN_HEAD: return launch<D, MQA_KV_FP8_E4M3_PER_TOKEN_HEAD>(a, stream);
        case MQA_KV_INT8_PER_TOKEN_HEAD: return launch<D, MQA_KV_INT8_PER_TOKEN_HEAD>(a, stream);
        case MQA_KV_INT4_PER_TOKEN_HEAD: return launch<D, MQA_KV_INT4_PER_TOKEN_HEAD>(a, stream);
        case MQA_KV_FP8_E4M3_BLOCK: return launch<D, MQA_KV_FP8_E4M3_BLOCK>(a, stream);
        default: return launch<D, MQA_KV_INT8_BLOCK>(a, stream);
    }
}

}  // namespace

cudaError_t gqa_append(const GqaAppendArgs& a, int D, int kv_dtype, cudaStream_t stream) {
    return D == 128 ? dispatch<128>(a, kv_dtype, stream) : dispatch<64>(a, kv_dtype, stream);
}

cudaError_t mla_append(const MlaAppendArgs& a, bool fp8, cudaStream_t stream) {
    const int groups = (a.R / 64 + 1 + a.H + kIter * 8 - 1) / (kIter * 8);
    const long long row_tasks = static_cast<long long>(a.t.tokens) * groups;
    const long long grid = (row_tasks + kWarps - 1) / kWarps;
    return launch_with_pdl(fp8 ? mla_append_kernel<true> : mla_append_kernel<false>, dim3(static_cast<unsigned>(grid)),
                           dim3(32 * kWarps), 0, stream, a, groups, row_tasks);
}

}  // namespace mqa

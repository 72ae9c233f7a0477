// Stage 1 of windowed / block-scaled GQA paged decode (see gqa_win.cuh for the
// plan).  For query row r and key t of its KV head
//   x_t = scale * s_k <q_r, K_t>,  out_r = sum_t e^{x_t - lse_r} s_v V_t,
//   lse_r = ln sum_t e^{x_t}
// with s_k, s_v the scales of the token block and head (1 for bf16).
//
// What bounds it: the bytes of the visible keys and values, read once (a
// row block of up to 16 rows does 8 multiply-adds per byte of bf16 cache and
// twice that per 8-bit byte, far below the tensor rate), and, with an 8-bit
// cache, the instructions that widen the codes.
//
// One thread block = up to 8 consumer warps + 1 producer warp, two blocks per
// SM for up to 8 rows.  The producer copies the K and then the V plane of a
// tile (16 TS tokens, all KV heads) into a ring of slots with 5D tensor
// copies whose box lands head after head, each head a dense tile of 16-token
// rows under the 128-byte (64-byte) swizzle, so ldmatrix over eight tokens is
// free of bank conflicts and nothing is padded.  Block scales ride along as
// 4-byte asynchronous copies counted on the same barrier.  Consumer warp w
// takes KV head w % Hkv and subtile w / Hkv of every tile.
//   * Tokens are the MMA's M dimension: S^T = K Q^T (16 tokens x 8 rows per
//     row group), O^T = V^T P^T (16 head dims x 8 rows).
//   * 8-bit codes stay codes in shared memory.  K: one ldmatrix gives a lane
//     four consecutive codes of a token; the reduction order inside a
//     16-wide step is permuted alike in Q.  V: ldmatrix.trans over byte
//     pairs gives a lane two head dims of two tokens; a byte permute makes
//     the two f16 pairs, so accumulator rows g and g + 8 are head dims 2g and
//     2g + 1 and V is never written back widened.
//   * Online softmax in base 2; the reference maximum moves only when a logit
//     exceeds it by more than 8, which a warp vote finds without reductions.
//     The numerators keep a reference of their own for x + log2(s_v): the
//     weights of P.V stay within the f16 range whatever the scales'
//     magnitude, and no rescaling of V is needed.
//   * Masked keys: their logits are replaced by -inf, and V bits of keys that
//     no row of the block sees are cleared in registers, so stale or non-finite
//     bytes never reach an accumulator (int8 codes are always finite).  Where
//     a key is seen by some rows only and its V holds an Inf or NaN, the rows
//     are summed apart.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gqa_win.cuh"

namespace mqa {
namespace win {

constexpr int kMaxSlots = 12;

template <int D, int KIND>
struct Cfg {
    static constexpr int kElt = KIND == kWinBf16 ? 2 : 1;
    static constexpr int kLine = D * kElt >= 128 ? 128 : D * kElt;  // bytes of one swizzled line
    static constexpr int kPanels = D * kElt / kLine;
    static constexpr int kSteps = D / 16;
    __host__ __device__ static int slot_bytes(int hkv, int ts) { return 16 * ts * hkv * D * kElt; }
};

// Row splits: a row block of more than 8 rows is shared by two sets of
// consumer warps of 8 rows each, in one thread block per SM (16 + 1 warps)
// instead of two (8 + 1 warps each).  The second set reads and widens the same
// tile again, but a warp then holds 8 rows' accumulators and 16 warps hide
// each other's latencies; 16 rows to a warp (168 registers, 8 warps per SM)
// measured 112 us where this takes 60 (32 requests x 4 positions, window
// 4096, e4m3 blocks).
__host__ __device__ constexpr int ctas(int rs) { return rs == 1 ? 2 : 1; }

struct Layout {
    int exch, scales, ok, bars, cum, total;  // the ring of slots comes first
};

template <int D, int KIND>
__host__ __device__ inline Layout layout(int hkv, int ts, int rs, int nslots, int vb, int batch) {
    Layout l;
    l.exch = nslots * Cfg<D, KIND>::slot_bytes(hkv, ts);
    // TS > 1: half of the consumer warps hand (O, m, r, l) to the other half
    l.scales = l.exch + (ts > 1 ? hkv * (ts / 2) * rs * (D / 16 * 4 + 6) * 128 : 0);
    l.ok = l.scales + nslots * 32;
    l.bars = l.ok + (nslots * 4 + 7) / 8 * 8;
    l.cum = l.bars + nslots * 16;
    l.total = l.cum + 4 * (vb + 1 + batch) + 1024;  // + alignment of the base
    return l;
}

__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, int y, int plane, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %2, %2, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(0), "r"(y), "r"(plane), "r"(smem_u32(bar))
        : "memory");
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

// 16 tokens x 32 e4m3 codes times 32 e4m3 x 8 rows.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int KIND>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (KIND == kWinBf16)
        mma_bf16_16816(d, a, b0, b1);
    else
        mma_f16(d, a, b0, b1);
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
// Four int8 codes -> the f16 pairs of bytes (0, 1) and (2, 3).
__device__ __forceinline__ uint2 widen_adjacent(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    return make_uint2(int8_pair(u, 0x4140), int8_pair(u, 0x4342));
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

// Four fp32 values as e4m3 codes (round to nearest), lowest byte first.
__device__ __forceinline__ uint32_t e4m3_word(const float (&x)[4]) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
    return r;
}

// Whether a word of V (two bf16 values or four e4m3 codes) holds an Inf or NaN.
template <int KIND>
__device__ __forceinline__ bool non_finite(uint32_t w) {
    if constexpr (KIND == kWinBf16) return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    const uint32_t x = w & 0x7f7f7f7fu;
    return (x & 0xffu) == 0x7fu || (x & 0xff00u) == 0x7f00u || (x & 0xff0000u) == 0x7f0000u ||
           (x & 0xff000000u) == 0x7f000000u;
}

// Walks the (virtual request, tile range) pieces of a unit.
struct Pieces {
    int p, p1, v, per_seq, done;
    int j0, j1, cur, whole;
    __device__ __forceinline__ void init(const int* cum, int vb, int units, int T, int g) {
        per_seq = units == 0;
        done = 0;
        p = p1 = 0;
        v = 0;
        if (per_seq) {
            v = g;
            return;
        }
        const int U = win_units(units, T);
        if (g >= U) return;
        p = static_cast<int>(static_cast<long long>(g) * T / U);
        p1 = static_cast<int>(static_cast<long long>(g + 1) * T / U);
        int lo = 0, hi = vb - 1;  // the last virtual request starting at or before p
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cum[mid] <= p)
                lo = mid;
            else
                hi = mid - 1;
        }
        v = lo;
    }
    // The next piece: tiles [j0, j1) of virtual request cur.
    __device__ __forceinline__ bool next(const int* cum) {
        if (per_seq) {
            if (done) return false;
            done = 1;
            cur = v;
            j0 = 0;
            j1 = cum[v + 1] - cum[v];
            whole = 1;
            return true;
        }
        if (p >= p1) return false;
        while (cum[v + 1] <= p) ++v;  // skip virtual requests without keys
        const int end = min(p1, cum[v + 1]);
        cur = v;
        j0 = p - cum[v];
        j1 = end - cum[v];
        whole = j0 == 0 && end == cum[v + 1];
        p = end;
        return true;
    }
};

// cum[0 .. vb]: exclusive prefix of the virtual requests' tile counts; lens:
// clamped lengths.  Every thread of the block calls it; returns the total.
__device__ __forceinline__ int build_prefix(const WinArgs& a, int* cum, int* lens) {
    const int vb = a.batch * a.rb;
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) lens[b] = win_len(a, b, a.status);
    __syncthreads();
    for (int v = threadIdx.x; v < vb; v += blockDim.x) {
        const int b = a.rb == 1 ? v : v / a.rb;
        cum[v + 1] = win_visible(a, v - b * a.rb, lens[b]).nt;
    }
    if (threadIdx.x == 0) cum[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        int running = 0;
        for (int base = 0; base < vb; base += 32) {
            const int i = base + static_cast<int>(threadIdx.x);
            int x = i < vb ? cum[i + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o);
                if (static_cast<int>(threadIdx.x) >= o) x += u;
            }
            if (i < vb) cum[i + 1] = running + x;
            running += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    return cum[vb];
}

// MULTI: more than one query position per request; RS: row splits.
template <int D, int KIND, int RS, bool MULTI>
__global__ void __launch_bounds__(32 * (8 * RS + 1), ctas(RS)) gqa_win_kernel(const __grid_constant__ WinArgs a) {
    using C = Cfg<D, KIND>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int Hkv = a.Hkv, TS = a.ts, NT = Hkv * TS, NC = NT * RS, nslots = a.nslots;
    const int vb = a.batch * a.rb;
    const Layout lay = layout<D, KIND>(Hkv, TS, RS, nslots, vb, a.batch);
    const int sbytes = C::slot_bytes(Hkv, TS);
    float* scale_s = reinterpret_cast<float*>(smem + lay.scales);  // [slot][subtile * Hkv + head]
    uint32_t* ok_s = reinterpret_cast<uint32_t*>(smem + lay.ok);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars);
    uint64_t* empty = full + nslots;
    int* cum = reinterpret_cast<int*>(smem + lay.cum);
    int* lens = cum + vb + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool scaled = KIND != kWinBf16 && a.kv_scales != nullptr;

    if (threadIdx.x == 0) {
        prefetch_tmap(&a.tmap);
        for (int s = 0; s < nslots; ++s) {
            mbar_init(&full[s], scaled ? 33 : 1);
            mbar_init(&empty[s], NC);
        }
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const int T = build_prefix(a, cum, lens);  // contains __syncthreads
    const int tt = 16 * TS;
    Pieces pc;
    pc.init(cum, vb, a.units, T, blockIdx.x);

    if (warp == NC) {
        // ------------------------------------------------------------ producer
        const int nbx = tt / a.box_tok;  // boxes per tile (1 .. 8), lane l < nbx copies box l
        const int bbytes = sbytes / nbx;
        const int per = 32 / nbx;  // tiles whose block ids one load of the warp holds
        const int lt = lane / nbx, lb = lane - lt * nbx;
        int slot = 0;
        uint32_t phase = 0;
        uint32_t used = 0, parity = 0;  // slots ever filled, and the parity of their last fill
        bool dead = false;
        while (!dead && pc.next(cum)) {
            const int b = a.rb == 1 ? pc.cur : pc.cur / a.rb;
            const WinVis vis = win_visible(a, pc.cur - b * a.rb, lens[b]);
            const int s_end = min(a.sinks, vis.hi);
            const int32_t* bt = a.block_table + static_cast<long long>(b) * a.max_blocks;
            // block id of box lb of tile j + lt, -1 where the box holds no visible key
            auto load_ids = [&](int j) {
                if (lt >= per || j + lt >= pc.j1) return -1;
                const int tok = vis.tile(j + lt) * tt + lb * a.box_tok;
                const bool need = tok < vis.hi && (tok + a.box_tok > vis.lo || tok < s_end);
                if (!need) return -1;
                const int id = __ldg(bt + tok / a.page);
                if (id < 0 || id >= a.num_blocks) {
                    report(a.status, MQA_ERR_DEVICE_CHECK);
                    return -1;
                }
                return id;
            };
            int ids = load_ids(pc.j0), next_ids = load_ids(pc.j0 + per);
            int base = pc.j0;
            for (int j = pc.j0; !dead && j < pc.j1; ++j) {
                if (j == base + per) {
                    base = j;
                    ids = next_ids;
                    next_ids = load_ids(base + per);
                }
                const int t0 = vis.tile(j) * tt;
                const int id = __shfl_sync(0xffffffffu, ids, ((j - base) * nbx + lane) & 31);
                const bool valid = lane < nbx && id >= 0;
                const uint32_t ok = __ballot_sync(0xffffffffu, valid);
                const int tok = t0 + lane * a.box_tok;  // of box `lane`
                // scale `lane`: subtile lane / Hkv, head lane % Hkv
                const int sub = lane / Hkv, stok = t0 + sub * 16;
                const int sbox = min(sub * 16 / a.box_tok, nbx - 1);
                const int sid = __shfl_sync(0xffffffffu, id, sbox);
                const bool has_scale = scaled && lane < NT && sid >= 0;
#pragma unroll
                for (int plane = 0; plane < 2; ++plane) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase ^ 1))) {
                        report(a.status, MQA_ERR_DEVICE_TIMEOUT);
                        dead = true;
                        break;
                    }
                    if (lane == 0) {
                        ok_s[slot] = ok;
                        mbar_arrive_expect_tx(&full[slot], __popc(ok) * bbytes);
                    }
                    __syncwarp();
                    if (valid)
                        tma_load_5d(smem + slot * sbytes + lane * bbytes, &a.tmap, tok % a.page, id * 2 + plane,
                                    &full[slot]);
                    if (scaled) {
                        if (has_scale)
                            cp_async_4(scale_s + slot * 8 + lane,
                                       a.kv_scales + ((static_cast<long long>(sid) * 2 + plane) * a.scale_groups +
                                                      (stok % a.page) / a.scale_block) * Hkv + (lane - sub * Hkv));
                        cp_async_arrive(&full[slot]);
                    }
                    used |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | (phase << slot);
                    if (++slot == nslots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        // no copy of this block may be in flight when it ends
        for (int s = 0; s < nslots; ++s)
            if ((used >> s) & 1u)
                if (!mbar_wait(&full[s], (parity >> s) & 1u)) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
        return;
    }

    // ------------------------------------------------------------- consumers
    const int g = lane >> 2, c = lane & 3;
    const int rs = RS == 1 ? 0 : warp / NT, wt = RS == 1 ? warp : warp - rs * NT;
    const int sub = wt / Hkv, kh = wt - sub * Hkv;
    const int box = sub * 16 / a.box_tok;
    // this warp's 16-token tile inside a slot, panel p at + p * panel_bytes
    const int panel_bytes = a.box_tok * C::kLine;
    const uint32_t tile = smem_u32(smem) + box * (sbytes / (tt / a.box_tok)) + kh * C::kPanels * panel_bytes +
                          (sub * 16 - box * a.box_tok) * C::kLine;
    // A lane's ldmatrix address of 16-byte chunks 2i, 2i + 1 of its row is
    // (row, chunk 0 or 1) with bit 5 + flipped by i: the swizzle only xors.
    // K (and 8-bit V) matrices are (tokens 0-7, chunk), (8-15, chunk),
    // (0-7, chunk + 1), (8-15, chunk + 1); bf16 V swaps the middle two.
    auto lane_at = [](int row, int ch) {
        if constexpr (C::kLine == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
        return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
    };
    const uint32_t k_at = tile + lane_at((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
    const uint32_t v_at =
        KIND == kWinBf16 ? tile + lane_at((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1) : k_at;
    constexpr int kPairs = C::kLine / 32;  // chunk pairs of one line

    int slot = 0;
    uint32_t phase = 0, slot_off = 0;
    bool aborted = false;
    // A wait that runs out is reported once; from then on the warp waits for
    // nothing and writes nothing, but still meets the other warps.
    auto wait_full = [&]() {
        if (aborted) return false;
        if (__all_sync(0xffffffffu, mbar_wait(&full[slot], phase))) return true;
        report(a.status, MQA_ERR_DEVICE_TIMEOUT);
        aborted = true;
        return false;
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0 && !aborted) mbar_arrive(&empty[slot]);
        slot_off += sbytes;
        if (++slot == nslots) {
            slot = 0;
            slot_off = 0;
            phase ^= 1;
        }
    };

    while (pc.next(cum)) {
        const int b = a.rb == 1 ? pc.cur : pc.cur / a.rb;
        const int rblk = pc.cur - b * a.rb;
        const WinVis vis = win_visible(a, rblk, lens[b]);
        const int row0 = rblk * 16 + rs * 8;
        // positions of this warp's first and last row, and the keys they see
        const int i_last = (min(a.rows, row0 + 8) - 1) / a.grp;
        const int p_first = MULTI ? vis.n - a.q_len + row0 / a.grp : vis.p_first;
        const int p_last = MULTI ? vis.n - a.q_len + i_last : vis.p_last;
        const int lo = p_first - a.window;  // the last key before the window of the first row
        const bool idle = RS > 1 && row0 >= a.rows;

        // Q^T operand (row g): bf16; f16 in the order of the int8 codes' words;
        // or two e4m3 terms of the row scaled by a power of two, q = f (q1 +
        // q2 / 16): 4 + 4 significant bits hold a bf16 value exactly, down to
        // 2^-21 of the row's largest entry
        uint32_t qb[C::kSteps][2];
        float qf[2] = {1.f, 1.f};  // f of rows 2c, 2c + 1 (e4m3)
        int qpos[2];               // positions of rows 2c, 2c + 1
        {
            const int R = row0 + g;
            const int i = MULTI ? R / a.grp : 0;
            const bool have = R < a.rows;
            const __nv_bfloat16* qr =
                a.q + ((static_cast<long long>(b) * a.q_len + i) * a.Hq + kh * a.grp + (R - i * a.grp)) * D;
            if constexpr (KIND == kWinBf16) {
#pragma unroll
                for (int ks = 0; ks < C::kSteps; ++ks) {
                    qb[ks][0] = have ? __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * c)) : 0u;
                    qb[ks][1] = have ? __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * c + 8)) : 0u;
                }
            } else {
                uint2 v[C::kSteps];  // entries 16 ks + 4c .. + 3
#pragma unroll
                for (int ks = 0; ks < C::kSteps; ++ks)
                    v[ks] = have ? __ldg(reinterpret_cast<const uint2*>(qr + ks * 16 + 4 * c)) : make_uint2(0u, 0u);
                if constexpr (KIND == kWinInt8) {
#pragma unroll
                    for (int ks = 0; ks < C::kSteps; ++ks) {
                        qb[ks][0] = q_f16(v[ks].x);
                        qb[ks][1] = q_f16(v[ks].y);
                    }
                } else {
                    float top = 0.f;
#pragma unroll
                    for (int ks = 0; ks < C::kSteps; ++ks) {
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[ks].x << 16)),
                                               fabsf(__uint_as_float(v[ks].x & 0xffff0000u))));
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[ks].y << 16)),
                                               fabsf(__uint_as_float(v[ks].y & 0xffff0000u))));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // 2^e above top; the row times 2^(8 - e) stays below 256
                    const int e = max(-100, static_cast<int>(__float_as_uint(top) >> 23) - 126);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - e) << 23);
                    const float f = __uint_as_float(static_cast<uint32_t>(127 - 8 + e) << 23);
                    qf[0] = __shfl_sync(0xffffffffu, f, 8 * c);  // of row 2c: any lane with g = 2c
                    qf[1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
                    for (int ks = 0; ks < C::kSteps; ++ks) {
                        float x[4] = {__uint_as_float(v[ks].x << 16) * up, __uint_as_float(v[ks].x & 0xffff0000u) * up,
                                      __uint_as_float(v[ks].y << 16) * up, __uint_as_float(v[ks].y & 0xffff0000u) * up};
                        const uint32_t hi = e4m3_word(x);
                        const uint32_t h01 = e4m3_pair(hi), h23 = e4m3_pair(hi >> 16);
                        const float2 f01 = __half22float2(bits_half2(h01)), f23 = __half22float2(bits_half2(h23));
                        x[0] = (x[0] - f01.x) * 16.f;
                        x[1] = (x[1] - f01.y) * 16.f;
                        x[2] = (x[2] - f23.x) * 16.f;
                        x[3] = (x[3] - f23.y) * 16.f;
                        qb[ks][0] = hi;
                        qb[ks][1] = e4m3_word(x);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int Re = min(row0 + 2 * c + e, a.rows - 1);
                qpos[e] = MULTI ? vis.n - a.q_len + Re / a.grp : vis.p_last;
            }
        }
        float o[C::kSteps][4];
        // references of the sums and (8-bit) of the numerators: base-2
        // exponents, and the logit above which they move (-inf: none yet)
        float m_ref[2] = {0.f, 0.f}, m_thr[2] = {-INFINITY, -INFINITY};
        float r_ref[2] = {0.f, 0.f}, r_thr[2] = {-INFINITY, -INFINITY};
        float l_part[2] = {0.f, 0.f};
#pragma unroll
        for (int mb = 0; mb < C::kSteps; ++mb) o[mb][0] = o[mb][1] = o[mb][2] = o[mb][3] = 0.f;

        for (int j = pc.j0; j < pc.j1; ++j) {
            const int t0 = vis.tile(j) * tt + sub * 16;
            float st[2][4];
            bool act = false;
            float ksc = a.sl2;
            if (wait_full()) {
                act = ((ok_s[slot] >> box) & 1u) && t0 <= p_last && (t0 + 15 > lo || t0 < a.sinks) && !idle;
                if (act) {
                    if (scaled) ksc *= scale_s[slot * 8 + wt];
                    const uint32_t kb = k_at + slot_off;
#pragma unroll
                    for (int e = 0; e < 2; ++e) st[e][0] = st[e][1] = st[e][2] = st[e][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < C::kPanels * kPairs; ++i) {
                        uint32_t w[4];
                        ldsm(w, ((kb + (i / kPairs) * panel_bytes) ^ ((i % kPairs) << 5)));
                        if constexpr (KIND == kWinBf16) {  // one 16-wide step
                            mma<KIND>(st[i & 1], w, qb[i][0], qb[i][1]);
                        } else if constexpr (KIND == kWinE4m3) {  // one 32-wide step, both terms of Q
                            mma_e4m3(st[0], w, qb[2 * i][0], qb[2 * i + 1][0]);
                            mma_e4m3(st[1], w, qb[2 * i][1], qb[2 * i + 1][1]);
                        } else {  // two 16-wide steps
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint2 k0 = widen_adjacent(w[2 * e]), k1 = widen_adjacent(w[2 * e + 1]);
                                const uint32_t af[4] = {k0.x, k1.x, k0.y, k1.y};
                                mma<KIND>(st[e], af, qb[2 * i + e][0], qb[2 * i + e][1]);
                            }
                        }
                    }
                }
            }
            release();
            const bool have_v = wait_full();
            if (act && have_v) {
                const float lvs = scaled ? log2f(scale_s[slot * 8 + wt]) : 0.f;
                // a tile at the edge of what the rows see: mask key by key
                const bool edge = t0 + 15 > p_first || (t0 + 15 >= a.sinks && t0 <= p_last - a.window);
                float x[4];  // token g: rows 2c, 2c + 1; token g + 8
                const float f0 = ksc * qf[0], f1 = ksc * qf[1];
                if constexpr (KIND == kWinE4m3) {
                    x[0] = fmaf(st[1][0], 0.0625f, st[0][0]) * f0;
                    x[1] = fmaf(st[1][1], 0.0625f, st[0][1]) * f1;
                    x[2] = fmaf(st[1][2], 0.0625f, st[0][2]) * f0;
                    x[3] = fmaf(st[1][3], 0.0625f, st[0][3]) * f1;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = (st[0][e] + st[1][e]) * ksc;
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = t0 + g + (e >> 1) * 8, p = qpos[e & 1];
                        if (!(t <= p && (t < a.sinks || t > p - a.window))) x[e] = -INFINITY;
                    }
                }
                bool grow = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mx = fmaxf(x[e], x[2 + e]);
                    grow |= mx > m_thr[e];
                    if (KIND != kWinBf16) grow |= mx + lvs > r_thr[e];
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[e], x[2 + e]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        float f = 1.f;
                        if (mx > m_thr[e]) {
                            f = m_thr[e] == -INFINITY ? 0.f : ex2(m_ref[e] - mx);
                            l_part[e] *= f;
                            m_ref[e] = mx;
                            m_thr[e] = mx + 8.f;
                        }
                        if (KIND != kWinBf16) {
                            f = 1.f;
                            mx += lvs;
                            if (mx > r_thr[e]) {
                                f = r_thr[e] == -INFINITY ? 0.f : ex2(r_ref[e] - mx);
                                r_ref[e] = mx;
                                r_thr[e] = mx + 8.f;
                            }
                        }
#pragma unroll
                        for (int mb = 0; mb < C::kSteps; ++mb) {
                            o[mb][e] *= f;
                            o[mb][2 + e] *= f;
                        }
                    }
                }
                // the sums take the fp32 probabilities; P.V takes them rounded
                uint32_t pb[2];
                {
                    const float p0 = ex2(x[0] - m_ref[0]), p1 = ex2(x[1] - m_ref[1]);
                    const float p2 = ex2(x[2] - m_ref[0]), p3 = ex2(x[3] - m_ref[1]);
                    l_part[0] += p0 + p2;
                    l_part[1] += p1 + p3;
                    if (KIND != kWinBf16) {
                        const float d0 = lvs - r_ref[0], d1 = lvs - r_ref[1];
                        pb[0] = movmatrix_t(p_pair<KIND>(ex2(x[0] + d0), ex2(x[1] + d1)));
                        pb[1] = movmatrix_t(p_pair<KIND>(ex2(x[2] + d0), ex2(x[3] + d1)));
                    } else {
                        pb[0] = movmatrix_t(p_pair<KIND>(p0, p1));
                        pb[1] = movmatrix_t(p_pair<KIND>(p2, p3));
                    }
                }
                const uint32_t vb_at = v_at + slot_off;
                // V words of tokens 2c, 2c + 1 (x) and + 8 (y): bits kept
                auto keep = [&](int p_min, int p_max) {
                    auto seen = [&](int t) { return t <= p_max && (t < a.sinks || t > p_min - a.window); };
                    const int t = t0 + 2 * c;
                    return make_uint2((seen(t) ? 0xffffu : 0u) | (seen(t + 1) ? 0xffff0000u : 0u),
                                      (seen(t + 8) ? 0xffffu : 0u) | (seen(t + 9) ? 0xffff0000u : 0u));
                };
                // operand A of head dims 16 mb ..: rows g and g + 8
                auto load_v = [&](int mb2, uint2 k, uint32_t (&av)[2][4]) {  // blocks 2 mb2, 2 mb2 + 1
                    if constexpr (KIND == kWinBf16) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = 2 * mb2 + e;
                            ldsm_t(av[e], (vb_at + (i / kPairs) * panel_bytes) ^ ((i % kPairs) << 5));
                            av[e][0] &= k.x;
                            av[e][1] &= k.x;
                            av[e][2] &= k.y;
                            av[e][3] &= k.y;
                        }
                    } else {
                        uint32_t w[4];
                        ldsm_t(w, vb_at ^ (mb2 << 5));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if constexpr (KIND == kWinE4m3) {
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
                const uint2 kp = edge ? keep(p_first, p_last) : make_uint2(~0u, ~0u);
                bool apart = false;
                if (MULTI && KIND != kWinInt8 && edge && p_first != p_last) {
                    // some key is seen by some rows only: is any V value Inf or NaN?
#pragma unroll
                    for (int i = 0; i < C::kPanels * kPairs; ++i) {
                        uint32_t w[4];
                        ldsm_t(w, (k_at + slot_off + (i / kPairs) * panel_bytes) ^ ((i % kPairs) << 5));
                        apart |= non_finite<KIND>(w[0] & kp.x) || non_finite<KIND>(w[1] & kp.y) ||
                                 non_finite<KIND>(w[2] & kp.x) || non_finite<KIND>(w[3] & kp.y);
                    }
                    apart = __any_sync(0xffffffffu, apart);
                }
                if (!MULTI || !apart) {
#pragma unroll
                    for (int mb2 = 0; mb2 < C::kSteps / 2; ++mb2) {
                        uint32_t av[2][4];
                        load_v(mb2, kp, av);
                        mma<KIND>(o[2 * mb2], av[0], pb[0], pb[1]);
                        mma<KIND>(o[2 * mb2 + 1], av[1], pb[0], pb[1]);
                    }
                } else {
                    for (int p = p_first; p <= p_last; ++p) {  // one query position at a time
                        const uint2 k1 = keep(p, p);
#pragma unroll
                        for (int mb2 = 0; mb2 < C::kSteps / 2; ++mb2) {
                            uint32_t av[2][4];
                            load_v(mb2, k1, av);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                mma<KIND>(d, av[e], pb[0], pb[1]);
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    if (qpos[y & 1] == p) o[2 * mb2 + e][y] += d[y];
                            }
                        }
                    }
                }
            }
            release();
        }

        // ---- the rows' sums over the warp's lanes, then over its subtiles;
        // references become -inf where there is none
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_part[e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            l_part[e] = l;
            if (m_thr[e] == -INFINITY) m_ref[e] = -INFINITY;
            if (KIND == kWinBf16)
                r_ref[e] = m_ref[e];
            else if (r_thr[e] == -INFINITY)
                r_ref[e] = -INFINITY;
        }
        if (TS > 1) {
            constexpr int kPerLane = C::kSteps * 4 + 6;
            float* exch = reinterpret_cast<float*>(smem + lay.exch);
            for (int half = TS / 2; half >= 1; half >>= 1) {
                float* buf = exch + ((rs * (TS / 2) + (sub & (half - 1))) * Hkv + kh) * kPerLane * 32 + lane;
                float* tail = buf + C::kSteps * 4 * 32;
                if (sub >= half && sub < 2 * half) {
#pragma unroll
                    for (int mb = 0; mb < C::kSteps; ++mb)
#pragma unroll
                        for (int y = 0; y < 4; ++y) buf[(mb * 4 + y) * 32] = o[mb][y];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        tail[e * 96] = m_ref[e];
                        tail[e * 96 + 32] = r_ref[e];
                        tail[e * 96 + 64] = l_part[e];
                    }
                }
                named_bar_sync(1, 32 * NC);
                if (sub < half) {
                    float f0[2], f1[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m1 = tail[e * 96], r1 = tail[e * 96 + 32], l1 = tail[e * 96 + 64];
                        const float m = fmaxf(m_ref[e], m1), r = fmaxf(r_ref[e], r1);
                        const float mu = m == -INFINITY ? 0.f : m, ru = r == -INFINITY ? 0.f : r;
                        l_part[e] = l_part[e] * ex2(m_ref[e] - mu) + l1 * ex2(m1 - mu);
                        f0[e] = ex2(r_ref[e] - ru);
                        f1[e] = ex2(r1 - ru);
                        m_ref[e] = m;
                        r_ref[e] = r;
                    }
#pragma unroll
                    for (int mb = 0; mb < C::kSteps; ++mb)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            o[mb][y] = o[mb][y] * f0[y & 1] + buf[(mb * 4 + y) * 32] * f1[y & 1];
                }
                named_bar_sync(1, 32 * NC);
            }
            if (sub > 0) continue;
        }
        if (aborted) continue;

        // ---- epilogue: rows 2c + e; head dims by kind (see the top)
        const int vslot = static_cast<int>(blockIdx.x) + pc.cur;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int jr = rs * 8 + 2 * c + e, R = rblk * 16 + jr;
            if (jr >= a.rbn || R >= a.rows) continue;
            const float l = l_part[e];
            // l == 0: no visible key (a NaN sum goes through to the output)
            float f = 0.f;
            if (l != 0.f) f = a.out_scale * (r_ref[e] == -INFINITY ? 0.f : ex2(r_ref[e] - m_ref[e])) / l;
            const float lse = l != 0.f ? (m_ref[e] + log2f(l)) * kLn2 : -INFINITY;
            if (pc.whole) {
                const int i = MULTI ? R / a.grp : 0;
                const long long orow =
                    (static_cast<long long>(b) * a.q_len + i) * a.Hq + kh * a.grp + (R - i * a.grp);
                __nv_bfloat16* op = a.out + orow * D;
#pragma unroll
                for (int mb = 0; mb < C::kSteps; ++mb) {
                    if constexpr (KIND == kWinBf16) {
                        op[mb * 16 + g] = __float2bfloat16_rn(o[mb][e] * f);
                        op[mb * 16 + g + 8] = __float2bfloat16_rn(o[mb][2 + e] * f);
                    } else {
                        *reinterpret_cast<uint32_t*>(op + mb * 16 + 2 * g) = pack_bf16x2(o[mb][e] * f, o[mb][2 + e] * f);
                    }
                }
                if (a.lse && g == 0) a.lse[orow] = lse;
            } else {
                const long long prow = (static_cast<long long>(vslot) * Hkv + kh) * a.rbn + jr;
                float* op = a.ws_o + prow * D;
#pragma unroll
                for (int mb = 0; mb < C::kSteps; ++mb) {
                    if constexpr (KIND == kWinBf16) {
                        op[mb * 16 + g] = o[mb][e] * f;
                        op[mb * 16 + g + 8] = o[mb][2 + e] * f;
                    } else {
                        *reinterpret_cast<float2*>(op + mb * 16 + 2 * g) = make_float2(o[mb][e] * f, o[mb][2 + e] * f);
                    }
                }
                if (g == 0) a.ws_lse[prow] = lse;
            }
        }
    }
}

template <int D, int KIND, int RS>
cudaError_t launch(WinArgs a, int grid, cudaStream_t stream) {
    const int vb = a.batch * a.rb;
    // dynamic shared memory of one block: 227 KB, or its share of the SM's 228 KB
    const int limit = ctas(RS) == 1 ? 227 * 1024 : 228 * 1024 / ctas(RS) - 1024;
    int ns = kMaxSlots;
    while (ns > 2 && layout<D, KIND>(a.Hkv, a.ts, RS, ns, vb, a.batch).total > limit) --ns;
    a.nslots = ns;
    const int bytes = layout<D, KIND>(a.Hkv, a.ts, RS, ns, vb, a.batch).total;
    auto kern = a.q_len > 1 ? gqa_win_kernel<D, KIND, RS, true> : gqa_win_kernel<D, KIND, RS, false>;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        e != cudaSuccess)
        return e;
    return launch_with_pdl(kern, dim3(grid), dim3(32 * (a.Hkv * a.ts * RS + 1)), bytes, stream, a);
}

template <int KIND>
cudaError_t dispatch(const WinArgs& a, int D, int grid, cudaStream_t stream) {
    if (D == 128)
        return a.rbn <= 8 ? launch<128, KIND, 1>(a, grid, stream) : launch<128, KIND, 2>(a, grid, stream);
    return a.rbn <= 8 ? launch<64, KIND, 1>(a, grid, stream) : launch<64, KIND, 2>(a, grid, stream);
}

}  // namespace win
}  // namespace mqa

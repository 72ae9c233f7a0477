// Attention of a ragged batch of new tokens over a paged GQA cache that holds
// their keys and values already (see gqa_prefill.cuh for cells and pieces).
// For the query row of a token at position p and query head h, over the keys t
// that it sees (t < max(p + 1, prefix), and t < sinks or t > p - window),
//   x_t = cap tanh(scale s_k <q, K_t> / cap) - slope_h |p - t|,
//   out = sum_t e^{x_t - lse} s_v V_t,   lse = ln sum_t e^{x_t}
// with s_k, s_v the scales of the token block and head (1 for bf16); no cap:
// the scaled product itself; no slopes: no bias.
//
// One thread block per multiprocessor.  Two tiles of 128 query rows share every
// block of 128 keys; roles by warp:
//   0-3, 4-7   softmax of tile 0 and 1: one row a thread
//   8          copies K and V blocks (tensor copies of box_tok tokens of one
//              head, 128-byte swizzle) into a ring
//   9          issues the tensor-core products: S_i = Q_i K^T (M = 128 rows, N =
//              128 keys) and O_i += P_i V, for the two tiles in turn, so that one
//              tile's softmax runs beside the other's products
//   10         walks the thread block's pieces, describes them for the others in a
//              ring in shared memory, and copies their queries
//   11 (8-bit caches: 12-15)  make blocks ready: clear V rows that no row of the cell sees
//              (whatever bytes they hold: 0 * NaN), and widen 8-bit codes to bf16
// TMEM (512 columns): O_0, O_1 (D fp32 columns each), S_0, S_1 (128 each); P_i
// (bf16) overwrites S_i.
//
// Softmax in base 2; a row's reference moves only when a logit exceeds it by
// more than 8 (P stays below 2^8, sums are fp32), so O is rarely rescaled, and
// the tile's own softmax warps do that.  P is rounded to bf16 for the tensor
// cores, the denominator sums the unrounded values.  8-bit codes widen to bf16
// exactly; K scales multiply the logits, V scales the numerators before they are
// rounded.
//
// What bounds it, measured on the prompts of perf/more_operators.py and changes of them
// (us a call, 12 calls in a row; 32/8 heads x 128 unless said).  One prompt of 15999
// tokens: 1315, the tensor cores (1595 TFLOP/s, 1627 where a call stands alone, of the 1952
// of a library's matrix product; a cell's start and end, and 4 % for looking V rows over
// for an Inf or NaN, are the rest).  Else the chain from product to softmax to product of
// each tile, as P lies where S did; where it was profiled no unit is full (64/8 heads x 64
// 2075: half the products for as many exponentials; slopes 1765, a cap of 50 1859, both
// 3198; e4m3 1716, block scales 2109, int8 64/8 x 64 2745, e4m3 with a cap 2602).  Blocks
// that take the slow form (see MODE below) take four to five times as long: caps of 20 and
// 15, which these logits of deviation 3 reach, 8533 and 8399, slopes up to 17 6028, a
// negative scale 6249.
// Short rows are bound by the starts and ends of cells and by masked edges: six prompts of
// 500 to 2600 tokens 122, 120 with a window of 1024 (10 blocks for 8 seen), capped at 50
// too 174, at 20 537.  Few tokens behind long contexts (three chunks of 64 behind 20 to 40
// thousand): 90, over e4m3 101, with slopes 114.
//
// Figures of steps below are of like batches: the prompt of 15999 tokens; six prompts of
// 522, 1400, 2600, 900, 1800 and 1500 tokens behind 3, 100, 50, 20, 0 and 77; three chunks
// of 64 behind 20, 30 and 40 thousand; 24 chunks of 1 to 700 tokens behind up to 900.
#pragma once

#include <atomic>
#include <type_traits>

#include "gqa_prefill.cuh"
#include "tc_ptx.cuh"

namespace mqa {
namespace pre {

enum Mode { kPlain, kCapped, kBiased, kBoth };

constexpr float kNone = -3e38f;  // reference before the first logit
// Below it a logit's factor could vanish beside a block's K scale (2^-100 at least), and a masked key's -inf times it be
// a NaN: such calls, and scales <= 0, multiply before they mask.
constexpr float kLeastScale = 0x1p-40f;

template <int D, int KIND>
struct Cfg {
    static constexpr bool kCodes = KIND != kWinBf16;
    static constexpr int kPanels = D / 64;                        // 64-column panels of a bf16 tile
    static constexpr int kPanel = kPreBlock * 128;                // bytes of one
    static constexpr int kTile = kPanels * kPanel;                // bytes of a bf16 tile of 128 rows
    static constexpr int kRaw = kCodes ? kPreBlock * D : 0;       // bytes of a block of codes
    static constexpr int kStages = kCodes ? (D == 128 ? 3 : 5) : (D == 128 ? 5 : 8);  // bf16 ring
    static constexpr int kRawStages = kCodes ? (D == 128 ? 4 : 6) : 0;
    static constexpr int kQ = D == 64 ? 2 : 1;  // cells whose queries are held
    static constexpr int kHelper = kCodes ? 12 : 11, kHelpers = kCodes ? 4 : 1;  // first of them, how many
    static constexpr int kThreads = 32 * (kHelper + kHelpers);
    // registers a thread: 64 K by the launch, moved between the warpgroups
    static constexpr int kRegsSoftmax = kCodes ? 200 : 216, kRegsRest = kCodes ? 56 : 72;
    static constexpr int kInfo = 8;  // blocks whose validity and scales are kept (at most 6 are between copy and softmax)
};

// A piece: blocks [j0, j1) of a cell's keys for one KV head (see PreCell).
struct Piece {
    int row0, cnt, p0, pre;
    int hi, lo, s_end, ns;
    int w0, nt, j0, j1;
    int b, h, more;  // more: 0 behind the last piece
    __device__ __forceinline__ int block(int j) const { return j < ns ? j : w0 + j - ns; }
};
constexpr int kPieces = 4;  // described ahead

// Tokens of a piece whose V row holds an Inf or NaN, in blocks that not every row of
// the cell sees all of: that row counts as zeros in the products (0 * NaN would reach
// the rows that do not see it), and the rows that see it become NaN at the end.
// The softmax of a tile reads them while blocks behind its last one, which it has not
// waited for, are still looked over: a block's tokens lie behind every row's limit
// until its first one is stored, and are not seen by the tile's rows after that.
struct BadTokens {
    int any;  // 1 where a bit below is set, 2 where there was no room for one
    int first[8];
    uint32_t bits[8][4];
    __device__ __forceinline__ void clear() {
        *this = {};
        for (int& t : first) t = kPreNoWindow;
    }
    // Row r of the piece's block number e of those looked over.
    __device__ __forceinline__ void found(int e, int r) {
        if (e < 8) atomicOr(&bits[e][r >> 5], 1u << (r & 31));
        atomicOr(&any, e < 8 ? 1 : 2);
    }
};

struct alignas(16) Shared {  // (what follows it is read 16 bytes at a time)
    uint64_t kv_full[8];   // copies landed (a raw stage's for codes)
    uint64_t kv_free[8];   // codes: read by the helpers; bf16: see ready / used
    uint64_t ready[8];     // a bf16 stage may be multiplied
    uint64_t used[8];      // .. and was
    uint64_t q_full[2], q_free[2];
    uint64_t piece_full[kPieces], piece_free[kPieces];
    uint64_t s_full[2], p_full[2], o_done[2], o_free[2], drain;
    long long scan[16];
    long long total;
    int b[2], u[2], h[2], j[2];  // start and end of the block's share
    uint32_t tmem;
    Piece piece[kPieces];
    BadTokens bad[kPieces];
    uint32_t valid[8];       // 16-token groups of a block that were copied
};
// What block-scaled caches have beside: K and V scales of the groups, logarithms and
// reciprocals of V's, and whether one of K's leaves 2^-100 .. 2^100, one of V's 2^-40 ..
// 2^40 (or is a NaN): such blocks are rare.
struct alignas(16) Extra {
    float scale[8][4][8];
    uint32_t far[8];
};

template <int D, int KIND>
constexpr int smem_bytes() {
    using C = Cfg<D, KIND>;
    return (2 * C::kQ + C::kStages) * C::kTile + C::kRawStages * C::kRaw + static_cast<int>(sizeof(Shared) + (C::kCodes ? sizeof(Extra) : 0));
}

__device__ __forceinline__ void tma_load(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_prefetch(const void* tmap, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(tmap), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void st_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}
// Two bf16 values times zero, added to sum.
__device__ __forceinline__ uint32_t times_zero(uint32_t v, uint32_t sum) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(sum));
    return d;
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(v));
    return v;
}
// Tensor-core products issued by the lane whose `on` is set.  The whole warp runs
// the code around them, converged (its waits end in a vote), so that descriptors
// stay in uniform registers: in a branch of one lane each product took 80 to 130
// cycles to issue, and a prompt of 15999 tokens 2323 us instead of 1745.
__device__ __forceinline__ void umma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
        : "memory");
}
__device__ __forceinline__ void umma_done(uint32_t on, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(on)
        : "memory");
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A wait of the whole warp, which is converged after it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

// ---- pairs of fp32 values, one instruction for both
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, "
        "%1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, "
        "%1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 "
        "w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Three-way maxima, of the values and of their magnitudes.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// cap2 tanh(y) / y by the polynomial c.
template <int N>
__device__ __forceinline__ float2 tanh_over(const float (&c)[N], float2 y) {
    const float2 z = mul2(y, y);
    float2 w = both(c[N - 1]);
#pragma unroll
    for (int k = N - 2; k >= 0; --k) w = fma2(w, z, both(c[k]));
    return w;
}
// One y = x / cap2, capped.
__device__ __forceinline__ float capped(const PreArgs& a, float y) {
    return fabsf(y) <= 1.f ? y * tanh_over(a.tanh_c, both(y)).x : tanh_far(a.cap2, y);
}

// ---- codes
__device__ __forceinline__ float2 half2_f32(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two codes, bytes 2 i and 2 i + 1 of w, as two fp32 values (exact).
template <int KIND, int I>
__device__ __forceinline__ float2 code_pair(uint32_t w) {
    if constexpr (KIND == kWinE4m3) {
        return half2_f32(e4m3x2_to_f16x2(I ? w >> 16 : w & 0xffffu));
    } else {
        // 2^23 + (code + 128) is exact in the mantissa of 0x4b000000
        const uint32_t u = w ^ 0x80808080u;
        return add2(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + 2 * I)),
                                __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441 + 2 * I))),
                    both(-8388736.f));
    }
}

// Walks the pieces of a thread block's share.
struct Pieces {
    PreReq req;
    PreCell cell;
    int b, u, h, j0, j1, cells;
    int eb, eu, eh, ej;
    int jn;  // first block of the next piece

    __device__ __forceinline__ void load(const PreArgs& a) {
        req = pre_request(a, b, nullptr);
        cells = (req.cnt + 2 * a.tile_tok - 1) / (2 * a.tile_tok);
    }
    __device__ __forceinline__ void init(const PreArgs& a, const Shared& s) {
        b = s.b[0];
        u = s.u[0];
        h = s.h[0] - 1;
        jn = s.j[0];
        eb = s.b[1];
        eu = s.u[1];
        eh = s.h[1];
        ej = s.j[1];
        if (b < a.batch) {
            load(a);
            cell = pre_cell(a, req, u);
        }
    }
    // The next piece: blocks [j0, j1) of cell (b, u), head h.
    __device__ __forceinline__ bool next(const PreArgs& a) {
        if (b >= a.batch) return false;
        if (++h == a.Hkv) {
            h = 0;
            if (++u >= cells) {
                u = 0;
                do {
                    if (++b >= a.batch) return false;
                    load(a);
                } while (cells == 0);
            }
            cell = pre_cell(a, req, u);
        }
        j0 = jn;
        jn = 0;
        const bool last = b == eb && u == eu && h == eh;
        if (last && ej == 0) return false;
        if (last || (b == eb && u == eu && h > eh) || (b == eb && u > eu) || b > eb) {
            if (!last) return false;
            j1 = ej;
            b = a.batch;  // nothing after it (cell, h and the fields above stay)
            return true;
        }
        j1 = cell.nt;
        return true;
    }
};

// The rows of tile i in a cell, and what they see.
struct TileView {
    int cnt;      // tokens
    int lo_first, lo_last, lim_first, lim_last;
    __device__ __forceinline__ TileView(const PreArgs& a, const Piece& c, int i) {
        const int t0 = i * a.tile_tok;
        cnt = min(a.tile_tok, c.cnt - t0);
        const int p0 = c.p0 + t0, p1 = p0 + cnt - 1;
        lo_first = p0 - a.window + 1;
        lo_last = p1 - a.window + 1;
        lim_first = p0 < 0 ? 0 : max(p0 + 1, c.pre);
        lim_last = p1 < 0 ? 0 : max(p1 + 1, c.pre);
    }
    // whether a row sees a key of the block from token t on
    __device__ __forceinline__ bool active(const PreArgs& a, int t) const {
        return cnt > 0 && t < lim_last && (t + kPreBlock > lo_first || t < a.sinks);
    }
    // whether every row sees all of it
    __device__ __forceinline__ bool whole(const PreArgs& a, int t) const {
        return t + kPreBlock <= lim_first && (t >= lo_last || t + kPreBlock <= a.sinks);
    }
};

__device__ __forceinline__ long long block_sum(Shared& s, long long v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s.scan[warp] = v;
    __syncthreads();
    long long t = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += s.scan[w];
    return t;
}
// Exclusive prefix over the block's threads; total in `all`.
__device__ __forceinline__ long long block_scan(Shared& s, long long v, long long& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s.scan[warp] = x;
    __syncthreads();
    long long before = 0, t = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
        if (w == warp) before = t;
        t += s.scan[w];
    }
    all = t;
    return before + x - v;
}

// The thread block's share: start and end in s.  Cuts inside a (cell, head) lie
// `grain` blocks apart, so that no piece is shorter than what a partial costs.
__device__ __forceinline__ void plan(const PreArgs& a, Shared& s, int* first) {
    const int tid = threadIdx.x, nthr = blockDim.x, c = blockIdx.x;
    // first[b]: cells of the requests before b
    long long before = 0;
    for (int base = 0; base < a.batch; base += nthr) {
        const int b = base + tid;
        int k = 0;
        if (b < a.batch) {
            const PreReq r = pre_request(a, b, c == 0 ? a.status : nullptr);
            k = a.cell_div(r.cnt + 2 * a.tile_tok - 1);
        }
        long long all;
        const long long at = before + block_scan(s, k, all);
        if (b < a.batch) first[b] = static_cast<int>(at);
        before += all;
    }
    // Requests that ascend have at most this many cells.  Starts that go down and up again can claim every token once
    // a request: far more work than the call's, and more cells than an int holds.  Nothing is done for them.
    if (before > a.num_tokens + a.batch) before = 0;
    if (tid < 2) {
        s.b[tid] = a.batch;
        s.u[tid] = s.h[tid] = s.j[tid] = 0;
    }
    __syncthreads();
    const int cells = static_cast<int>(before);
    auto find = [&](int i, int& b, int& u, int& nt) {
        int lo = 0, hi = a.batch - 1;  // the last request whose cells begin at or before i (empty ones lie before)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
        u = i - first[lo];
        nt = pre_cell(a, pre_request(a, b, nullptr), u).nt;
    };
    long long w = 0;
    for (int i = tid; i < cells; i += nthr) {
        int b, u, nt;
        find(i, b, u, nt);
        w += nt + a.cell_cost;
    }
    const long long total = block_sum(s, w) * a.Hkv;
    const long long share = total / a.grid;
    const int grain = !a.cut ? 1 << 30 : share >= 32 ? 1 : share >= 8 ? 2 : 4;
    const long long x[2] = {total * c / a.grid, total * (c + 1) / a.grid};
    long long base = 0;
    for (int i0 = 0; i0 < cells && base <= x[1]; i0 += nthr) {
        const int i = i0 + tid;
        int b = 0, u = 0, nt = 0;
        if (i < cells) find(i, b, u, nt);
        const int per = i < cells ? nt + a.cell_cost : 0;
        long long all;
        const long long at = base + block_scan(s, static_cast<long long>(per) * a.Hkv, all);
        base += all;
        for (int e = 0; e < 2; ++e) {
            if (per == 0 || x[e] < at || x[e] >= at + static_cast<long long>(per) * a.Hkv || (e == 1 && c + 1 == a.grid)) continue;
            int h = static_cast<int>((x[e] - at) / per);
            const int y = static_cast<int>(x[e] - at - static_cast<long long>(h) * per);
            // the nearest cut: a multiple of the grain, or an end
            int j = max(0, y - a.cell_cost);
            if (grain >= nt)
                j = 2 * y <= per ? 0 : nt;
            else
                j = (j + grain / 2) / grain * grain;
            int cb = b, cu = u;
            if (j > 0 && j + (grain + 1) / 2 >= nt) {  // the start of what follows
                j = 0;
                if (++h == a.Hkv) {
                    h = 0;
                    ++cu;  // past the request's last cell: normalised below
                }
            }
            s.b[e] = cb;
            s.u[e] = cu;
            s.h[e] = h;
            s.j[e] = j;
        }
        __syncthreads();
    }
    __syncthreads();
    if (tid == 0) {
        for (int e = 0; e < 2; ++e)
            while (s.b[e] < a.batch) {
                const int k = (s.b[e] + 1 < a.batch ? first[s.b[e] + 1] : cells) - first[s.b[e]];
                if (s.u[e] < k) break;
                ++s.b[e];
                s.u[e] = 0;
            }
        if (s.b[0] == s.b[1] && s.u[0] == s.u[1] && s.h[0] == s.h[1] && s.j[0] == s.j[1]) s.b[0] = a.batch;  // nothing
    }
    __syncthreads();
}

__device__ __forceinline__ float2 get2(const uint32_t (&x)[32], int e) {
    return make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
}
__device__ __forceinline__ void put2(uint32_t (&x)[32], int e, float2 v) {
    x[e] = __float_as_uint(v.x);
    x[e + 1] = __float_as_uint(v.y);
}
// Values whose bit is not set become v.
__device__ __forceinline__ void keep(uint32_t (&x)[32], uint32_t bits, float v) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!((bits >> e) & 1u)) x[e] = __float_as_uint(v);
}
// The largest value of each 16 (whose bit is set).
__device__ __forceinline__ float2 group_max(const uint32_t (&x)[32], uint32_t bits) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; ++e) top[e / 16] = fmaxf(top[e / 16], (bits >> e) & 1u ? __uint_as_float(x[e]) : -INFINITY);
    return make_float2(top[0], top[1]);
}
__device__ __forceinline__ float2 group_max(const uint32_t (&x)[32]) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 2) top[e / 16] = max3(top[e / 16], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
    return make_float2(top[0], top[1]);
}
__device__ __forceinline__ float chunk_max(const uint32_t (&x)[32]) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 2) top[e / 2 & 1] = max3(top[e / 2 & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
    return fmaxf(top[0], top[1]);
}

// y[32] := cap2 tanh(y), eight polynomials at a time.
template <int N>
__device__ __forceinline__ void cap_chunk(const float (&c)[N], uint32_t (&x)[32]) {
    constexpr int kChains = 8;
#pragma unroll
    for (int e = 0; e < 32; e += 2 * kChains) {
        float2 z[kChains], w[kChains];
#pragma unroll
        for (int k = 0; k < kChains; ++k) {
            z[k] = mul2(get2(x, e + 2 * k), get2(x, e + 2 * k));
            w[k] = fma2(z[k], both(c[N - 1]), both(c[N - 2]));
        }
#pragma unroll
        for (int q = N - 3; q >= 0; --q)
#pragma unroll
            for (int k = 0; k < kChains; ++k) w[k] = fma2(w[k], z[k], both(c[q]));
#pragma unroll
        for (int k = 0; k < kChains; ++k) put2(x, e + 2 * k, mul2(get2(x, e + 2 * k), w[k]));
    }
}

// Logits (base 2) of 32 keys from their products, whatever the shaping: times sl2
// and the scales f of the two groups of 16, capped (mid: all within the reach of
// kTanh), less slope2 |d - e|; -inf where `bits` has no bit.
__device__ __forceinline__ void shape_any(const PreArgs& a, uint32_t (&x)[32], float2 f, bool mid, float slope2, int d, uint32_t bits) {
    const bool cap = a.cap2 > 0.f;
    const float unit = cap ? a.sl2 * a.inv_cap2 : a.sl2;
#pragma unroll
    for (int e = 0; e < 32; e += 2) put2(x, e, mul2(get2(x, e), both(unit * (e < 16 ? f.x : f.y))));
    if (cap && mid) cap_chunk(a.tanh_c, x);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        float y = __uint_as_float(x[e]);
        if (cap && !mid) y = capped(a, y);
        x[e] = __float_as_uint(fmaf(-slope2, fabsf(static_cast<float>(d - e)), y));
    }
    keep(x, bits, -INFINITY);
}

// P of 32 keys as bf16 pairs from x f + add, a scale f for each 16 of them, and +
// slope2 e for key e if BIAS.  Their sum is added to l.  With TIMES P is multiplied by
// V's scales v of the two groups (codes are V's operand then, so that there is one
// rounding, of P v: bf16 has the range of any scale): by adding their logarithms before
// the exponential, and the sums of each 16 are multiplied by the reciprocals.
template <bool BIAS, bool TIMES>
__device__ __forceinline__ void numerators(const uint32_t (&x)[32], float2 f, float add, float slope2, float2 log_v, float2 rcp_v, float2 (&l)[2], uint32_t (&p)[16]) {
    float2 group = both(0.f);
    const float2 start = TIMES ? make_float2(add + log_v.x, add + log_v.y) : both(add);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float2 y = fma2(get2(x, 2 * k), both(k < 8 ? f.x : f.y), both(k < 8 ? start.x : start.y));
        if (BIAS) y = make_float2(fmaf(slope2, 2.f * k, y.x), fmaf(slope2, 2.f * k + 1.f, y.y));
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        if (TIMES)
            group = k % 8 == 0 ? e : add2(group, e);
        else
            l[k & 1] = add2(l[k & 1], e);
        p[k] = pack_bf16x2(e.x, e.y);
        if (TIMES && k % 8 == 7) l[k >> 3] = fma2(group, both(k < 8 ? rcp_v.x : rcp_v.y), l[k >> 3]);
    }
}
// The same of finished logits less their reference, multiplied by v as it is.
__device__ __forceinline__ void numerators_times(const uint32_t (&x)[32], float add, float2 v, float2 (&l)[2], uint32_t (&p)[16]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float2 y = add2(get2(x, 2 * k), both(add));
        float2 e = make_float2(ex2(y.x), ex2(y.y));
        l[k & 1] = add2(l[k & 1], e);
        e = mul2(e, both(k < 8 ? v.x : v.y));
        p[k] = pack_bf16x2(e.x, e.y);
    }
}

// 32 bytes, in one store where `wide` says that they are aligned to it.
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// O's columns of a warp's rows times f.
template <int D>
__device__ __forceinline__ void rescale(uint32_t o_at, float f) {
#pragma unroll 1
    for (int k = 0; k < D; k += 16) {
        uint32_t o[16];
        tmem_ld16(o_at + k, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st16(o_at + k, o);
    }
}

// Four lanes' rows of 128 bytes, v[8 u ..] the 32 bytes u of the lane's own row: after
// it v[8 j ..] are bytes 32 q .. of row j of the four, q = lane % 4.
__device__ __forceinline__ void transpose4(uint32_t (&v)[32]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
    for (int u = 0; u < 4; u += 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t x = v[8 * u + e], y = v[8 * u + 8 + e];
            const uint32_t z = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
            v[8 * u + e] = odd ? z : x;
            v[8 * u + 8 + e] = odd ? y : z;
        }
    // now pairs of rows: v[0 ..], v[8 ..] bytes 32 (q & 1) .., v[16 ..], v[24 ..] bytes 64 + 32 (q & 1) ..
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint32_t x = v[e], y = v[16 + e];
        const uint32_t z = __shfl_xor_sync(0xffffffffu, high ? x : y, 2);
        v[e] = high ? z : x;
        v[16 + e] = high ? y : z;
    }
}

// A row's D columns of O (at TMEM o_at) times f: bf16 to row orow of out, or a
// partial's fp32 to row prow; row < 0: nowhere.  f == 0: zeros, whatever O holds.
// The whole warp calls it.  Four lanes write whole lines of their rows in turn: what
// bounds the stores is their number of requests (32 bytes of 32 rows a store took
// 4500 cycles a tile).  (Four warps of their own for it kept the next cell's first
// products waiting longer than the softmax did: 148 and 168 us, by rows and by lines,
// where this takes 137, six prompts with a window of 1024.)
template <int D>
__device__ __forceinline__ void write_rows(const PreArgs& a, uint32_t o_at, bool part, float f, long long row) {
    const int q = threadIdx.x & 3;
    const bool wide = (reinterpret_cast<uintptr_t>(part ? static_cast<void*>(a.ws_o) : a.out) & 31) == 0;
    long long to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = __shfl_sync(0xffffffffu, row, (threadIdx.x & 28) + j);
    if (part) {
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
            uint32_t o[32];
            tmem_ld32(o_at + k, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = f == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * f);
            transpose4(o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t v[8] = {o[8 * j], o[8 * j + 1], o[8 * j + 2], o[8 * j + 3], o[8 * j + 4], o[8 * j + 5], o[8 * j + 6], o[8 * j + 7]};
                if (to[j] >= 0) st_global32(a.ws_o + to[j] * D + k + 8 * q, v, wide);
            }
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < D; k += 64) {
            uint32_t v[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t o[32];
                tmem_ld32(o_at + k + 32 * h, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[16 * h + e] = f == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
            }
            transpose4(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w[8] = {v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3], v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]};
                if (to[j] >= 0) st_global32(a.out + to[j] * D + k + 16 * q, w, wide);
            }
        }
    }
}

// A bf16 block's rows at the edges of what the cell sees, by one warp.  If `some`:
// rows that no row of the cell sees become zeros; if lim < hi: rows that some see and
// some do not, [lim, hi) and [lo, lo_last), are looked over for an Inf or NaN.
template <int D>
__device__ __forceinline__ void edge_rows(BadTokens& bad, int edge, uint32_t dst, uint32_t groups, int t0, int hi, int lo, int se, bool some,
                                       int lim, int lo_last) {
    // 16-byte chunks of rows from r0 to r1, a lane each (the swizzle only permutes a row's chunks)
    constexpr int kChunks = D / 8, kRows = 32 / kChunks;  // chunks of a row, rows at a time
    const int lane = threadIdx.x & 31, my_row = lane / kChunks;
    const uint32_t my_at = dst + ((lane % kChunks) >> 3) * (kPreBlock * 128) + (lane & 7) * 16;
    bool wrote = some;
    auto clear = [&](int r0, int r1) {
        for (int r = max(r0, 0) + my_row; r < min(r1, kPreBlock); r += kRows) st_zero16(my_at + r * 128);
    };
    if (some) {
        if (groups == 0xffu) {
            clear(hi - t0, kPreBlock);
            clear(se - t0, lo - t0);
        } else {
            for (int r = my_row; r < kPreBlock; r += kRows) {
                const int t = t0 + r;
                if (!(((groups >> (r >> 4)) & 1u) && t < hi && (t >= lo || t < se))) st_zero16(my_at + r * 128);
            }
        }
        __syncwarp();
    }
    auto look = [&](int r0, int r1) {
        // 0 times an Inf or NaN is a NaN, which stays in the sum
        uint32_t sum[4] = {0u, 0u, 0u, 0u};
        r0 = max(r0, 0) + my_row;
        r1 = min(r1, kPreBlock);
#pragma unroll 1
        for (int r = r0; r < r1; r += 4 * kRows) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = r + u * kRows < r1 ? ld_shared16(my_at + (r + u * kRows) * 128) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                sum[0] = times_zero(v[u].x, sum[0]);
                sum[1] = times_zero(v[u].y, sum[1]);
                sum[2] = times_zero(v[u].z, sum[2]);
                sum[3] = times_zero(v[u].w, sum[3]);
            }
        }
        if (!__any_sync(0xffffffffu, (sum[0] | sum[1] | sum[2] | sum[3]) != 0)) return;
        wrote = true;
        for (int r = r0; r < r1; r += kRows) {
            // an exponent of ones in a half of a word carries into its sign
            auto full = [](uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
            const uint4 v = ld_shared16(my_at + r * 128);
            if ((full(v.x) | full(v.y) | full(v.z) | full(v.w)) != 0) {
                bad.found(edge, r);
                st_zero16(my_at + r * 128);
            }
        }
    };
    if (lim < INT32_MAX) {
        look(lim - t0, hi - t0);
        look(lo - t0, lo_last - t0);
    }
    if (wrote) fence_proxy_async_smem();
}

// NaN where a row that sees t < lim, t >= lo or t < sinks sees one of the tokens, else 0.
static __device__ __noinline__ float bad_tokens(const BadTokens& bad, int lim, int lo, int sinks) {
    bool sees = (bad.any & 2) && lim > 0;
    for (int e = 0; e < 8; ++e)
        for (int k = 0; k < 4; ++k)
            for (uint32_t bits = bad.bits[e][k]; bits; bits &= bits - 1) {
                const int t = bad.first[e] + 32 * k + __ffs(bits) - 1;
                sees |= t < lim && (t >= lo || t < sinks);
            }
    return sees ? NAN : 0.f;
}

// The keys of a block that a row sees, relative to the block's first one: key e where e <
// lim and (e >= lo or e < sinks), if its group of 16 was copied.
struct Seen {
    int lim, lo, sinks;
    uint32_t groups;
    // of keys 32 k ..: bit e for key 32 k + e
    __device__ __forceinline__ uint32_t bits(int k) const {
        auto below = [](int e) { return e <= 0 ? 0u : e >= 32 ? 0xffffffffu : (1u << e) - 1u; };
        const int t = 32 * k;
        return below(lim - t) & (~below(lo - t) | below(sinks - t)) &
               (((groups >> (2 * k)) & 1u ? 0xffffu : 0u) | ((groups >> (2 * k + 1)) & 1u ? 0xffff0000u : 0u));
    }
};

// -inf in a row's products of keys that it does not see.  A function of its own, like
// rare_row, for the edges of what rows see.
static __device__ __noinline__ void mask_row(uint32_t s_at, int lim, int lo, int sinks, uint32_t groups) {
    const Seen seen = {lim, lo, sinks, groups};
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        uint32_t x[32];
        tmem_ld32(s_at + 32 * k, x);
        tmem_wait_ld();
        keep(x, seen.bits(k), -INFINITY);
        tmem_st32(s_at + 32 * k, x);
    }
    tmem_wait_st();
}

// A row's softmax of one block whatever the shaping, in chunks through TMEM: the
// logits take S's place, then P theirs (that of chunk k in columns 16 k .. 16 k + 15,
// of chunks that were read before).  A function of its own, so that its code lies
// apart from what usually runs.
struct RareRow {
    uint32_t s_at, o_at;    // the row's warp's S and O
    const float* scales;    // [2][8], of K's and V's groups, or null
    Seen seen;              // keys that count
    float slope2;
    int d;                  // distance of the first key
    bool mid, rescale;      // as of shape_any; whether O holds anything yet
    float m, l[2];          // reference and sum, in and out
    uint64_t* o_done;       // O's last product, and its phase
    int o_phase;
    float f;                // out: what other sums of the row are to be multiplied by
};
template <int D, bool TIMES>
__device__ __noinline__ bool rare_row(const PreArgs& a, RareRow& q) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        uint32_t y[32];
        tmem_ld32(q.s_at + 32 * k, y);
        tmem_wait_ld();
        shape_any(a, y, q.scales ? make_float2(q.scales[2 * k], q.scales[2 * k + 1]) : both(1.f), q.mid, q.slope2, q.d - 32 * k, q.seen.bits(k));
        mx = fmaxf(mx, chunk_max(y));
        tmem_st32(q.s_at + 32 * k, y);
    }
    tmem_wait_st();
    const bool move = mx > q.m + 8.f;
    q.f = move && q.rescale ? ex2(q.m - mx) : 1.f;
    if (move) q.m = mx;
    float2 l[2] = {make_float2(q.l[0] * q.f, q.l[1] * q.f), both(0.f)};
    if (q.rescale && __any_sync(0xffffffffu, move)) {
        if (!warp_wait(q.o_done, q.o_phase)) return false;
        tc_fence_after();
        rescale<D>(q.o_at, q.f);
    }
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        uint32_t y[32], o[16];
        tmem_ld32(q.s_at + 32 * k, y);
        tmem_wait_ld();
        float2 v = both(1.f);
        if (TIMES && q.scales) {
            const uint32_t bits = q.seen.bits(k);
            v = make_float2(bits & 0xffffu ? q.scales[8 + 2 * k] : 0.f, bits >> 16 ? q.scales[8 + 2 * k + 1] : 0.f);
        }
        numerators_times(y, -q.m, v, l, o);
        tmem_st16(q.s_at + 16 * k, o);
    }
    q.l[0] = l[0].x + l[1].x;
    q.l[1] = l[0].y + l[1].y;
    return true;
}

// SCALED: whether token blocks have scales (they cost a per-tensor cache with slopes
// 22 %: 154 us instead of 126, three chunks of 64 tokens).  MODE: kPlain (a scale that is no
// smaller than kLeastScale), kCapped, kBiased (slopes, or another scale), kBoth.  All keep
// a row's 128 products in registers; what is rare (a product beyond 0.6 of its cap in any
// row of a warp, a scale far below the cap, keys behind the query under slopes, steep
// biases, scales <= 0) is shaped in a loop of its own through TMEM, four to five times as
// slow, so that the code that runs stays short: with every case in line a capped prompt of
// 15999 tokens took 3509 us, a biased one 3728, a third of it waits for instructions.
template <int D, int KIND, bool SCALED, int MODE>
__global__ void __launch_bounds__(Cfg<D, KIND>::kThreads, 1) gqa_prefill_kernel(const __grid_constant__ PreArgs a) {
    using C = Cfg<D, KIND>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t q_s = smem_u32(smem), kv_s = q_s + 2 * C::kQ * C::kTile, raw_s = kv_s + C::kStages * C::kTile;
    Shared& s = *reinterpret_cast<Shared*>(smem + (2 * C::kQ + C::kStages) * C::kTile + C::kRawStages * C::kRaw);
    Extra& ex = *reinterpret_cast<Extra*>(&s + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr bool kCap = MODE == kCapped || MODE == kBoth, kBias = MODE == kBiased || MODE == kBoth;
    constexpr int kCopyStages = C::kCodes ? C::kRawStages : C::kStages;

    if (threadIdx.x == 0) {
        prefetch_tmap(&a.q_map);
        prefetch_tmap(&a.kv_map);
        for (int i = 0; i < 8; ++i) {
            mbar_init(&s.kv_full[i], SCALED ? 9 : 1);
            mbar_init(&s.kv_free[i], C::kHelpers);
            mbar_init(&s.ready[i], C::kHelpers);
            mbar_init(&s.used[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_free[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 128);
            mbar_init(&s.o_done[i], 1);
            mbar_init(&s.o_free[i], 4);

        }
        mbar_init(&s.drain, 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&s.piece_full[i], 1);
            mbar_init(&s.piece_free[i], 2 + C::kHelpers + 8);  // the warps that read it
        }
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&s.tmem, 512);
    pdl_wait();
    pdl_launch_dependents();
    plan(a, s, reinterpret_cast<int*>(smem + 2 * C::kQ * C::kTile));  // the ring is not in use yet
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    const uint32_t t_o = tmem, t_s = tmem + 2 * D;  // tile i: t_o + i D, t_s + 128 i

    bool ok = true;
    // Piece number n, once it is described; null behind the last one (or where the wait ran out).  The whole warp calls
    // it, and every wait below but those of warp 10's lane: code after them meets at full masks, so that a warp's lanes
    // have to give up together.
    auto piece = [&](int n) -> const Piece* {
        const Piece* pc = &s.piece[n % kPieces];
        if (!warp_wait(&s.piece_full[n % kPieces], n / kPieces & 1)) {
            ok = false;
            return nullptr;
        }
        return pc->more ? pc : nullptr;
    };
    auto piece_done = [&](int n) { mbar_arrive(&s.piece_free[n % kPieces]); };

    if (warp == 8) {
        // ------------------------------------------------ copies of K and V
        set_regs_down<C::kRegsRest>();
        const int nb = kPreBlock / a.box_tok, per = a.box_tok / 16;
        int kvc = 0;  // blocks of K or V copied
        for (int n = 0; ok; ++n) {
            const Piece* pp = piece(n);
            if (!pp) break;
            const Piece pc = *pp;
            if (pc.b == a.withhold) break;
            const int32_t* table = a.block_table + static_cast<long long>(pc.b) * a.max_blocks;
            // lane k < nb: box k of a block; its block id is fetched a block ahead
            auto want = [&](int j, int& off) {
                const int t = pc.block(j) * kPreBlock + lane * a.box_tok;
                if (lane >= nb || t >= pc.hi || !(t + a.box_tok > pc.lo || t < pc.s_end)) return -1;
                const int page = a.page_div(t);
                off = t - page * a.page;
                const int id = __ldg(table + page);
                return id < 0 || id >= a.num_blocks ? -2 : id;
            };
            int off = 0, off_next = 0, id_next = pc.j0 < pc.j1 ? want(pc.j0, off_next) : -1;
            for (int j = pc.j0; j < pc.j1 && ok; ++j) {
                const int id = id_next;
                off = off_next;
                if (j + 1 < pc.j1) id_next = want(j + 1, off_next);
                if (id == -2) report(a.status, MQA_ERR_DEVICE_CHECK);
                const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                uint32_t groups = 0xffu;
                if (have != (1u << nb) - 1u) {
                    groups = 0;
                    for (int k = 0; k < nb; ++k)
                        if ((have >> k) & 1u) groups |= ((1u << per) - 1u) << (k * per);
                }
                int g_id = 0, g_off = 0;
                if (SCALED) {
                    g_id = __shfl_sync(0xffffffffu, id, lane / per);
                    g_off = __shfl_sync(0xffffffffu, off, lane / per) + lane % per * 16;
                }
                const int slot = (kvc >> 1) % C::kInfo;
                for (int plane = 0; plane < 2; ++plane, ++kvc) {
                    const int st = kvc % kCopyStages;
                    uint64_t* free = C::kCodes ? &s.kv_free[st] : &s.used[st];
                    if (!warp_wait(free, (kvc / kCopyStages & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        if (plane == 0) s.valid[slot] = groups;
                        mbar_arrive_expect_tx(&s.kv_full[st], __popc(have) * a.box_tok * D * (C::kCodes ? 1 : 2));
                    }
                    __syncwarp();
                    if (id >= 0) {
                        const int row = id * 2 * a.page + plane * a.page + off;
                        if constexpr (C::kCodes) {
                            tma_load(raw_s + st * C::kRaw + lane * a.box_tok * D, &a.kv_map, 0, pc.h, row, &s.kv_full[st]);
                        } else {
#pragma unroll
                            for (int p = 0; p < C::kPanels; ++p)
                                tma_load(kv_s + st * C::kTile + p * C::kPanel + lane * a.box_tok * 128, &a.kv_map, p * 64, pc.h, row,
                                         &s.kv_full[st]);
                        }
                    }
                    if (SCALED && lane < 8) {
                        // (V's with K's: the softmax wants both)
                        if (plane == 0 && g_id >= 0) {
                            const float* from = a.kv_scales + (static_cast<long long>(g_id * 2) * a.scale_groups + a.scale_div(g_off)) * a.Hkv + pc.h;
                            cp_async_4(&ex.scale[slot][0][lane], from);
                            cp_async_4(&ex.scale[slot][1][lane], from + a.scale_groups * a.Hkv);
                            cp_async_arrive(&s.kv_full[st]);
                        } else {
                            if (plane == 0) ex.scale[slot][0][lane] = ex.scale[slot][1][lane] = 1.f;
                            mbar_arrive(&s.kv_full[st]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) piece_done(n);
        }
        if (!ok) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
        // no copy may be in flight at the end
        for (int q = max(kvc - kCopyStages, 0); q < kvc; ++q)
            if (!mbar_wait(&s.kv_full[q % kCopyStages], q / kCopyStages & 1)) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
    } else if (warp == 10) {
        // ------------------------------------------------ pieces and queries
        set_regs_down<C::kRegsRest>();
        if (lane == 0) {
            Pieces pw;
            pw.init(a, s);
            int queries = 0, head = 3, begun = 0, row0 = 0, cnt = 0, h = 0;
            // queries of the last described piece with blocks, not copied yet: a piece is
            // described (and its queries fetched towards L2) before the one before it gets
            // its queries, which waits for the products of the one before that
            int q_row = 0, q_cnt = 0, q_head = 0;
            auto copy_queries = [&]() {
                if (q_cnt == 0) return;
                const int qs = queries % C::kQ;
                if (queries >= C::kQ && !mbar_wait(&s.q_free[qs], (queries / C::kQ & 1) ^ 1)) {
                    ok = false;
                    return;
                }
                const int tiles = q_cnt > a.tile_tok ? 2 : 1;
                mbar_arrive_expect_tx(&s.q_full[qs], tiles * a.tile_rows * D * 2);
                for (int i = 0; i < tiles; ++i)
                    for (int p = 0; p < C::kPanels; ++p)
                        tma_load(q_s + (2 * qs + i) * C::kTile + p * C::kPanel, &a.q_map, p * 64, q_head * a.grp, q_row + i * a.tile_tok,
                                 &s.q_full[qs]);
                ++queries;
                q_cnt = 0;
            };
            for (int n = 0; ok; ++n) {
                const bool more = pw.next(a);
                if (n >= kPieces && !mbar_wait(&s.piece_free[n % kPieces], (n / kPieces & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                Piece& pc = s.piece[n % kPieces];
                const PreCell& c = pw.cell;
                s.bad[n % kPieces].clear();
                pc = {c.row0, c.cnt, c.p0, c.pre, c.hi, c.lo, c.s_end, c.ns, c.w0, c.nt, pw.j0, pw.j1, pw.b < a.batch ? pw.b : pw.eb, pw.h, more};
                mbar_arrive(&s.piece_full[n % kPieces]);
                const bool blocks = more && pw.j1 > pw.j0;
                if (more) {
                    if (n == 0) head = pw.j0 == 0 ? 0 : pw.j1 < c.nt ? 2 : 1;
                    begun = pw.j0 == 0 && pw.j1 < c.nt;
                    row0 = c.row0;
                    cnt = c.cnt;
                    h = pw.h;
                }
                if (blocks && queries > 0)
                    for (int i = 0; i < (cnt > a.tile_tok ? 2 : 1); ++i)
                        for (int p = 0; p < C::kPanels; ++p) tma_prefetch(&a.q_map, p * 64, h * a.grp, row0 + i * a.tile_tok);
                // The queries held back, whatever this piece is: over pieces without blocks they would be waited for
                // by a piece whose place in the ring is wanted next.  (In one place: copied in three, 24 chunks over int8
                // blocks took 280 us instead of 271.)
                for (bool held = !blocks;; held = true) {
                    copy_queries();
                    if (held || !ok) break;
                    q_row = row0;
                    q_cnt = cnt;
                    q_head = h;
                    if (queries > 0) break;
                }
                if (!more) break;
            }
            if (!ok) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
            for (int q = max(queries - C::kQ, 0); q < queries; ++q)  // no copy may be in flight at the end
                if (!mbar_wait(&s.q_full[q % C::kQ], q / C::kQ & 1)) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
            if (a.cut) {
                a.ws_meta[2 * blockIdx.x] = make_int4(begun, head, row0, cnt);
                a.ws_meta[2 * blockIdx.x + 1] = make_int4(h, 0, 0, 0);
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------ tensor-core products
        set_regs_down<C::kRegsRest>();
        constexpr uint32_t kIdQK = umma_idesc_bf16(128, kPreBlock, 0), kIdPV = umma_idesc_bf16(128, D, 1);
        const uint64_t qd = umma_desc(q_s, 16, 1024), kd = umma_desc(kv_s, 16, 1024), vd = umma_desc(kv_s, C::kPanel, 1024);
        const uint32_t on = elect_lane();
        int st = 0, ph = 0;          // stage and phase of the next K or V block that is waited for
        int qn = 0, qs = 0;          // pieces with blocks, where the queries of this one lie
        uint32_t pn0 = 0, pn1 = 0;   // P blocks of each tile
        uint32_t on0 = 0, on1 = 0;   // pieces with a product of each tile
        auto wait_block = [&](int& at) {  // the next K or V block
            at = st;
            ok = warp_wait(&s.ready[st], ph);
            if (++st == C::kStages) {
                st = 0;
                ph ^= 1;
            }
            tc_fence_after();
        };
        auto qk = [&](int i, int at) {
            const uint64_t aq = qd + static_cast<uint64_t>(((2 * qs + i) * C::kTile) >> 4), bk = kd + static_cast<uint64_t>((at * C::kTile) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t o = static_cast<uint64_t>(((k >> 2) * C::kPanel + (k & 3) * 32) >> 4);
                umma_ss(on, t_s + i * 128, aq + o, bk + o, kIdQK, k > 0);
            }
            umma_done(on, &s.s_full[i]);
        };
        auto pv = [&](int i, int at, bool begun) {
            const uint64_t bv = vd + static_cast<uint64_t>((at * C::kTile) >> 4);
#pragma unroll
            for (int k = 0; k < kPreBlock / 16; ++k)
                umma_ts(on, t_o + i * D, t_s + i * 128 + k * 8, bv + static_cast<uint64_t>((k * 16 * 128) >> 4), kIdPV, begun || k > 0);
            umma_done(on, &s.o_done[i]);
        };
        for (int n = 0; ok; ++n) {
            const Piece* pp = piece(n);
            if (!pp) break;
            const Piece pc = *pp;
            __syncwarp();
            if (lane == 0) piece_done(n);
            __syncwarp();
            if (pc.j1 <= pc.j0) continue;
            const TileView v0(a, pc, 0), v1(a, pc, 1);
            qs = qn % C::kQ;
            ok = warp_wait(&s.q_full[qs], qn++ / C::kQ & 1);
            if (!ok) break;
            uint32_t act = 0, begun = 0;  // tiles that the block has to do with; tiles with a product in this piece
            // P V of a block and Q K^T of the next one, tile by tile, so that one tile's
            // softmax runs beside the other's products
#pragma unroll 1
            for (int j = pc.j0 - 1; j < pc.j1 && ok; ++j) {
                const bool have = j >= pc.j0, more = j + 1 < pc.j1;
                const int t = more ? pc.block(j + 1) * kPreBlock : 0;
                const uint32_t next = more ? (v0.active(a, t) ? 1u : 0u) | (v1.active(a, t) ? 2u : 0u) : 0u;
                int kst = 0, vst = 0;
                if (have) wait_block(vst);
                if (!ok) break;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    if ((act >> i) & 1u) {
                        const uint32_t pn = i ? pn1++ : pn0++;
                        ok = warp_wait(&s.p_full[i], pn & 1u);
                        if (ok && !((begun >> i) & 1u)) {
                            const uint32_t n_o = i ? on1++ : on0++;
                            if (n_o > 0) ok = warp_wait(&s.o_free[i], (n_o - 1) & 1u);
                        }
                        if (!ok) break;
                        tc_fence_after();
                        pv(i, vst, (begun >> i) & 1u);
                        begun |= 1u << i;
                    }
                    if (more) {
                        if (i == 0) wait_block(kst);
                        if (!ok) break;
                        if ((next >> i) & 1u) qk(i, kst);
                    }
                }
                if (!ok) break;
                if (have) umma_done(on, &s.used[vst]);
                if (more) umma_done(on, &s.used[kst]);
                if (j + 2 == pc.j1) umma_done(on, &s.q_free[qs]);
                act = next;
            }
        }
        if (!ok) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
        // no product may be in flight at the end
        umma_done(on, &s.drain);
        if (!mbar_wait(&s.drain, 0)) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
    } else if (warp >= C::kHelper) {
        // ------------------------------------------------ making blocks ready
        set_regs_down<C::kRegsRest>();
        const int w = warp - C::kHelper;
        int kvc = 0;
        for (int n = 0; ok; ++n) {
            const Piece* pp = piece(n);
            if (!pp) break;
            const Piece pc = *pp;
            // what some rows of the cell see and some do not: [lim, hi) and [lo, lo_last)
            const int lim = pc.p0 < 0 ? 0 : max(pc.p0 + 1, pc.pre), lo_last = pc.p0 + pc.cnt - a.window;
            BadTokens& bad = s.bad[n % kPieces];
            int edges = 0;
            for (int j = pc.j0; j < pc.j1 && ok; ++j) {
                const int t0 = pc.block(j) * kPreBlock, hi = pc.hi, lo = pc.lo, se = pc.s_end;
                for (int plane = 0; plane < 2; ++plane, ++kvc) {
                    const int st = kvc % C::kStages, rst = kvc % kCopyStages, slot = (kvc >> 1) % C::kInfo;
                    if (!__all_sync(0xffffffffu, mbar_wait(&s.kv_full[rst], kvc / kCopyStages & 1) &&
                                                     (!C::kCodes || mbar_wait(&s.used[st], (kvc / C::kStages & 1) ^ 1)))) {
                        ok = false;
                        break;
                    }
                    if (SCALED && plane == 0 && w == 0) {
                        // (a K scale of 0, whose codes are 0: their products stay 0, and -inf where nothing is seen stays that)
                        float k = 1.f, v = 1.f;
                        if (lane < 8) {
                            k = ex.scale[slot][0][lane];
                            v = ex.scale[slot][1][lane];
                            if (k >= 0.f && k < 0x1p-100f) ex.scale[slot][0][lane] = k = 0x1p-100f;
                            ex.scale[slot][2][lane] = log2f(v);
                            ex.scale[slot][3][lane] = 1.f / v;
                        }
                        const uint32_t far = __any_sync(0xffffffffu, !(k >= 0x1p-100f && k <= 0x1p100f && v >= 0x1p-40f && v <= 0x1p40f));
                        if (lane == 0) ex.far[slot] = far;
                    }
                    const uint32_t groups = s.valid[slot];
                    const bool all = groups == 0xffu && t0 + kPreBlock <= hi && (t0 >= lo || t0 + kPreBlock <= se);
                    // V rows that not every row of the cell sees are looked over
                    const bool look = plane == 1 && KIND != kWinInt8 &&
                                      ((t0 < hi && t0 + kPreBlock > lim && lim < hi) || (t0 < lo_last && t0 + kPreBlock > lo && lo < lo_last));
                    const int edge = edges;
                    if (look) {
                        ++edges;
                        if (edge < 8 && w == 0 && lane == 0) bad.first[edge] = t0;
                    }
                    auto seen = [&](int r) {
                        const int t = t0 + r;
                        return ((groups >> (r >> 4)) & 1u) && t < hi && (t >= lo || t < se);
                    };
                    const uint32_t dst = kv_s + st * C::kTile;
                    if constexpr (!C::kCodes) {
                        if (__builtin_expect(look || ((plane == 1 || kCap) && !all), 0))
                            edge_rows<D>(bad, edge, dst, groups, t0, hi, lo, se, !all, look ? lim : INT32_MAX, lo_last);
                    } else {
                        // a lane takes 16 codes of row r: chunk q of the raw row, two chunks of the wide one.  How many at
                        // a time: where this bounds the block, four (e4m3 without scales or a cap: 1707 us where two take 1876, one
                        // prompt of 15999 tokens); else two, as short code counts (capped 2539 where four take 2817, 24 chunks over
                        // int8 blocks 229 and 243); at edges one (six prompts with a window over e4m3 184, four 211)
                        constexpr int kQ4 = D / 64, kUnits = kPreBlock / 8 * kQ4 / C::kHelpers, kAtOnce = kCap || SCALED ? 2 : 4;
                        const uint32_t src = raw_s + rst * C::kRaw;
                        auto widen = [&](auto whole) {
#pragma unroll 1
                            for (int u0 = 0; u0 < kUnits; u0 += decltype(whole)::value ? kAtOnce : 1) {
                                constexpr int kAt = decltype(whole)::value ? kAtOnce : 1;
                                uint4 c[kAt];
#pragma unroll
                                for (int u = 0; u < kAt; ++u) {
                                    const int i = (u0 + u) * C::kHelpers + w, r = i / kQ4 * 8 + (lane & 7), q = i % kQ4 * 4 + (lane >> 3);
                                    const uint32_t at = D == 128 ? r * 128 + ((q ^ (r & 7)) << 4) : r * 64 + ((q ^ ((r >> 1) & 3)) << 4);
                                    c[u] = decltype(whole)::value || seen(r) ? ld_shared16(src + at) : make_uint4(0, 0, 0, 0);
                                    if (!decltype(whole)::value && look) {  // (e4m3: a NaN's seven ones carry into the sign)
                                        auto full = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
                                        if ((full(c[u].x) | full(c[u].y) | full(c[u].z) | full(c[u].w)) != 0) {
                                            bad.found(edge, r);
                                            c[u] = make_uint4(0, 0, 0, 0);
                                        }
                                    }
                                }
#pragma unroll
                                for (int u = 0; u < kAt; ++u) {
                                    const int i = (u0 + u) * C::kHelpers + w, r = i / kQ4 * 8 + (lane & 7), q = i % kQ4 * 4 + (lane >> 3);
                                    const uint32_t in[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
                                    uint32_t o[8];
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float2 x = code_pair<KIND, 0>(in[k]), y = code_pair<KIND, 1>(in[k]);
                                        o[2 * k] = pack_bf16x2(x.x, x.y);
                                        o[2 * k + 1] = pack_bf16x2(y.x, y.y);
                                    }
                                    const uint32_t row = dst + (q >> 2) * C::kPanel + r * 128;
                                    const int ch = (q & 3) * 2;
                                    st_shared16(row + ((ch ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
                                    st_shared16(row + (((ch + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
                                }
                            }
                        };
                        if (look || ((plane == 1 || kCap) && !all))
                            widen(std::false_type{});
                        else
                            widen(std::true_type{});
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&s.ready[st]);
                        if (C::kCodes) mbar_arrive(&s.kv_free[rst]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) piece_done(n);
        }
        if (!ok) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
    } else if (warp == 11) {
        set_regs_down<C::kRegsRest>();  // (with its warpgroup)
    } else {
        // ------------------------------------------------ softmax of tile i
        set_regs_up<C::kRegsSoftmax>();
        const int i = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t my_s = t_s + i * 128 + lanes, my_o = t_o + i * D + lanes;
        const int tk = a.grp_div(r), g = r - tk * a.grp;  // token of the tile, head of the group
        int sn = 0, kvb = 0;  // blocks of this tile, of the thread block
        for (int n = 0; ok; ++n) {
            const Piece* pc = piece(n);
            if (!pc) break;
            const TileView view(a, *pc, i);
            const int p = pc->p0 + i * a.tile_tok + tk;
            const bool row = tk < view.cnt && r < a.tile_rows;
            const int lim = row && p >= 0 ? max(p + 1, pc->pre) : 0, lo = p - a.window + 1;
            float slope2 = 0.f;
            if (kBias && a.slopes && row) slope2 = __ldg(a.slopes + pc->h * a.grp + g) * kLog2e;
            // where a bias falls by more than 64 over 32 keys (or rises), rows take the largest logit itself
            const bool steep = kBias && __any_sync(0xffffffffu, !(slope2 >= 0.f && slope2 * 31.f <= 64.f));
            float m = kNone;
            float2 l[2] = {both(0.f), both(0.f)};
            int nact = 0;
            const int j1 = pc->j1;
            for (int j = pc->j0; j < j1; ++j, ++kvb) {
                const int t0 = pc->block(j) * kPreBlock;
                if (!view.active(a, t0)) continue;
                if (!warp_wait(&s.s_full[i], sn & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t groups = s.valid[kvb % C::kInfo];
                const bool edge = groups != 0xffu || !view.whole(a, t0);
                // (a block may lie 2^30 before a row's window and more: relative positions do not leave the range)
                const Seen seen = {lim - t0, lo - t0, a.sinks - t0, groups};
                uint32_t x[4][32];
                float4 ks[2] = {make_float4(1.f, 1.f, 1.f, 1.f), make_float4(1.f, 1.f, 1.f, 1.f)};
                if (SCALED && !kCap) {
                    ks[0] = *reinterpret_cast<const float4*>(&ex.scale[kvb % C::kInfo][0][0]);
                    ks[1] = *reinterpret_cast<const float4*>(&ex.scale[kvb % C::kInfo][0][4]);
                }
                auto scales = [&](int k) {  // of the two groups of chunk k (with a cap from shared memory: registers)
                    if (kCap && SCALED) return make_float2(ex.scale[kvb % C::kInfo][0][2 * k], ex.scale[kvb % C::kInfo][0][2 * k + 1]);
                    return k & 1 ? make_float2(ks[k >> 1].z, ks[k >> 1].w) : make_float2(ks[k >> 1].x, ks[k >> 1].y);
                };
                if (!kCap && __builtin_expect(edge, 0)) mask_row(my_s, seen.lim, seen.lo, seen.sinks, seen.groups);
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(my_s + 32 * k, x[k]);
                tmem_wait_ld();
                // Logarithms and reciprocals of V's scales of the two groups of chunk k (the row's keys of groups that
                // it does not see are -inf, whatever is added)
                auto v_scales = [&](int k, int which) {
                    return SCALED ? *reinterpret_cast<const float2*>(&ex.scale[kvb % C::kInfo][which][2 * k]) : both(0.f);
                };
                // The row's reference after a block whose largest logit is mx (or less); false if a wait ran out.
                auto refer = [&](float mx) {
                    const bool move = mx > m + 8.f;
                    if (nact == 0) {
                        if (move) m = mx;
                    } else if (__any_sync(0xffffffffu, move)) {
                        float f = 1.f;
                        if (move) {
                            f = ex2(m - mx);
                            m = mx;
                        }
                        l[0] = mul2(l[0], both(f));
                        l[1] = mul2(l[1], both(f));
                        // the product before must be in O
                        if (!warp_wait(&s.o_done[i], (sn - 1) & 1)) return false;
                        tc_fence_after();
                        rescale<D>(my_o, f);
                    }
                    return true;
                };
                // (scales of 0, infinite ones and NaN reach the rows that see a key of theirs)
                bool rare = SCALED && ex.far[kvb % C::kInfo] != 0, mid = false;
                if constexpr (kCap) {
                    float size = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float wide[2] = {0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            wide[e / 16] = max3_abs(wide[e / 16], __uint_as_float(x[k][e]), __uint_as_float(x[k][e + 1]));
                        const float2 f = scales(k);
                        size = max3(size, wide[0] * f.x, wide[1] * f.y);
                    }
                    size *= fabsf(a.sl2) * a.inv_cap2;  // (a NaN passes the comparisons of the others and stays one)
                    rare |= a.tiny_unit || __any_sync(0xffffffffu, row && size > 0.6f);
                    mid = !__any_sync(0xffffffffu, row && size > 1.f);
                }
                if constexpr (kBias) rare |= steep || (pc->pre > 0 && t0 + kPreBlock > pc->p0 + i * a.tile_tok);
                if constexpr (kCap || kBias) rare |= !(a.sl2 >= kLeastScale);
                if (__builtin_expect(rare, 0)) {
                    RareRow q = {my_s, my_o, SCALED ? &ex.scale[kvb % C::kInfo][0][0] : nullptr, seen, slope2, p - t0, mid, nact > 0, m,
                                 {l[0].x, l[0].y}, &s.o_done[i], (sn - 1) & 1};
                    ok = rare_row<D, SCALED>(a, q);
                    m = q.m;
                    l[1] = mul2(l[1], both(q.f));
                    l[0] = make_float2(q.l[0], q.l[1]);
                } else {
                    float b[4];
                    // Masked keys' -inf stay that under the cap: its leading coefficient is positive.
                    // (kBoth masks maxima and capped logits in registers: with the call bf16 spills, 4743
                    // us for one prompt of 15999 tokens where it takes 3207; with -inf put in before the
                    // maxima bf16 takes 2681, but e4m3 5157 where it takes 3681.)
                    if (kCap && !kBias && __builtin_expect(edge, 0)) {
                        mask_row(my_s, seen.lim, seen.lo, seen.sinks, seen.groups);
#pragma unroll
                        for (int k = 0; k < 4; ++k) tmem_ld32(my_s + 32 * k, x[k]);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (kCap && kBias && edge) {
                            const float2 f = scales(k), top = group_max(x[k], seen.bits(k));
                            b[k] = fmaxf(top.x * f.x, top.y * f.y);
                        } else if constexpr (SCALED) {
                            const float2 f = scales(k), top = group_max(x[k]);
                            b[k] = fmaxf(top.x * f.x, top.y * f.y);
                        } else {
                            b[k] = chunk_max(x[k]);
                        }
                    }
                    float mx;
                    if constexpr (kBias) {
                        // Instead of the largest logit a bound of it: the largest product of
                        // each 32 keys less the bias of the nearest (at most 64 too large, see
                        // `steep`; numerators of 2^-64 lose nothing in bf16 or fp32).
                        const float d = static_cast<float>(p - t0);  // distance of the block's first key
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            b[k] *= a.sl2;
                            if (kCap && b[k] > -INFINITY) b[k] = b[k] * a.inv_cap2 * tanh_over(a.tanh_near, both(b[k] * a.inv_cap2)).x;
                            b[k] = fmaf(-slope2, fmaxf(0.f, d - (32.f * k + 31.f)), b[k]);
                        }
                        mx = max3(fmaxf(b[0], b[1]), b[2], b[3]);
                    } else {
                        mx = max3(fmaxf(b[0], b[1]), b[2], b[3]) * a.sl2;
                        if (kCap && mx > -INFINITY) mx = mx * a.inv_cap2 * tanh_over(a.tanh_near, both(mx * a.inv_cap2)).x;
                    }
                    ok = refer(mx);
                    if constexpr (kCap) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (SCALED) {
                                const float2 f = scales(k);
#pragma unroll
                                for (int e = 0; e < 32; e += 2) put2(x[k], e, mul2(get2(x[k], e), both(e < 16 ? f.x : f.y)));
                            } else if (KIND == kWinE4m3 && !kBias) {
                                if (a.raw_unit != 1.f) {
#pragma unroll
                                    for (int e = 0; e < 32; e += 2) put2(x[k], e, mul2(get2(x[k], e), both(a.raw_unit)));
                                }
                            }
                            cap_chunk(a.tanh_raw, x[k]);
                        }
                        if (kBias && edge) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) keep(x[k], seen.bits(k), -INFINITY);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[16];
                        float2 f = both(a.sl2);
                        if constexpr (kCap)
                            f = both(1.f);
                        else if constexpr (SCALED)
                            f = mul2(scales(k), both(a.sl2));
                        // With a bias: every key that is seen lies at or before the query, slope2 e -
                        // slope2 d (a row sees its own key at distance 0, beside which the rounding
                        // of a far key's bias is nothing).
                        const float add = kBias ? fmaf(-slope2, static_cast<float>(p - t0 - 32 * k), -m) : -m;
                        numerators<kBias, SCALED>(x[k], f, add, slope2, v_scales(k, 2), v_scales(k, 3), l, o);
                        tmem_st16(my_s + 16 * k, o);
                    }
                }
                if (!ok) break;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&s.p_full[i]);
                ++sn;
                ++nact;
            }
            if (!ok) break;
            // ---- the piece's result
            if (nact > 0 && !warp_wait(&s.o_done[i], (sn - 1) & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float sum = l[0].x + l[0].y + l[1].x + l[1].y;
            if (__builtin_expect(s.bad[n % kPieces].any != 0, 0)) sum += bad_tokens(s.bad[n % kPieces], lim, lo, a.sinks);
            const int j0 = pc->j0;
            const bool part = j0 > 0 || j1 < pc->nt;
            const long long orow = static_cast<long long>(pc->row0 + i * a.tile_tok + tk) * a.Hq + pc->h * a.grp + g;
            const long long prow = (2LL * blockIdx.x + (j0 > 0 ? 0 : 1)) * kPreSlotRows + i * kPreTile + r;
            // sum == 0: no visible key (a NaN goes through to the output)
            const float f = sum == 0.f ? 0.f : part ? a.out_scale : a.out_scale / sum;
            if (row) {
                if (part) {
                    *reinterpret_cast<float2*>(a.ws_ml + 2 * prow) = make_float2(sum == 0.f ? -INFINITY : m, sum);
                } else if (a.lse) {
                    a.lse[orow] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
                }
            }
            write_rows<D>(a, my_o, part, f, !row ? -1 : part ? prow : orow);
            __syncwarp();
            if (lane == 0) piece_done(n);
            if (nact > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.o_free[i]);
            }
        }
        if (!ok) report(a.status, MQA_ERR_DEVICE_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int KIND, bool SCALED, int MODE>
cudaError_t launch(const PreArgs& a, cudaStream_t stream) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    constexpr int bytes = smem_bytes<D, KIND>();
    static_assert(bytes <= 227 * 1024, "shared memory");
    auto kern = gqa_prefill_kernel<D, KIND, SCALED, MODE>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (!known || !done[dev].load(std::memory_order_relaxed)) {
        if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); e != cudaSuccess) return e;
        if (known) done[dev].store(true, std::memory_order_relaxed);
    }
    return launch_with_pdl(kern, dim3(a.grid), dim3(Cfg<D, KIND>::kThreads), bytes, stream, a);
}

template <int KIND, bool SCALED, int MODE>
cudaError_t dispatch_size(const PreArgs& a, int D, cudaStream_t stream) {
    return D == 128 ? launch<128, KIND, SCALED, MODE>(a, stream) : launch<64, KIND, SCALED, MODE>(a, stream);
}

template <int KIND, bool SCALED>
cudaError_t dispatch(const PreArgs& a, int D, cudaStream_t stream) {
    if (a.cap2 > 0.f)
        return a.slopes ? dispatch_size<KIND, SCALED, kBoth>(a, D, stream) : dispatch_size<KIND, SCALED, kCapped>(a, D, stream);
    if (a.slopes || !(a.sl2 >= kLeastScale)) return dispatch_size<KIND, SCALED, kBiased>(a, D, stream);
    return dispatch_size<KIND, SCALED, kPlain>(a, D, stream);
}

}  // namespace pre
}  // namespace mqa

// Windowed and block-scaled GQA paged decode: arguments, the visible-key plan
// of the stage-1 kernels, and the host interface.
//
// A request's query rows (q_len positions x the query heads of a KV head) are
// cut into row blocks of up to 24; request and row block together are one
// "virtual request" v = b * rb + r with its own keys.  The query at position p sees
// key t iff  t <= p and (t < sinks or t > p - window), so the keys of a row
// block are the sinks [0, min(sinks, hi)) and the run [lo, hi), where hi is
// its last position + 1 and lo = max(0, first position - window + 1).  They
// are walked in tiles of `tt` consecutive tokens; the tiles of all virtual
// requests are laid end to end and cut into units of about equal size, one
// per thread block, so only tiles that hold a visible key are ever read.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace mqa {

// Cache formats of the kernels.
enum WinKind { kWinBf16 = 0, kWinE4m3 = 1, kWinInt8 = 2 };

constexpr int kWinMaxVirtual = 2048;  // virtual requests whose tile prefix fits in shared memory
constexpr int kWinNoWindow = 1 << 30;  // windows from here on are none
// .. and the kernels take this one: beyond every position (lengths are at most
// INT32_MAX - 1024), and a position, -128 at least, minus it is an int
constexpr int kWinUnbounded = INT32_MAX - 1024;

// Exact division of 0 <= n < 2^31 by a divisor known on the host: with l =
// ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n)
// >> l (Granlund and Montgomery, "Division by invariant integers").
struct FastDiv {
    uint32_t m, l;
    static FastDiv of(int d) {
        uint32_t l = 0;
        while ((1ull << l) < static_cast<uint64_t>(d)) ++l;
        return {static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - static_cast<uint64_t>(d))) / static_cast<uint64_t>(d) + 1), l};
    }
    __device__ __forceinline__ int operator()(int n) const {
        return static_cast<int>((__umulhi(m, static_cast<uint32_t>(n)) + static_cast<uint32_t>(n)) >> l);
    }
};

struct WinArgs {
    CUtensorMap tmap;  // {line, rows (block, plane, token), panels, heads}
    const __nv_bfloat16* q;   // [batch, q_len, Hq, D]
    const float* kv_scales;   // [blocks, 2, page / scale_block, Hkv], or null: no block scales
    const int32_t* block_table;
    const int32_t* seq_lens;
    __nv_bfloat16* out;
    float* lse;
    float* ws_o;    // [slots, Hkv, rbn, D], normalised partials
    float* ws_lse;  // [slots, Hkv, rbn]
    int2* ws_units; // [batch * rb]: first and last unit of each virtual request
    int* status;
    float sl2;        // scale * log2(e) (times k_scale of a per-tensor e4m3 cache)
    float out_scale;  // v_scale of a per-tensor e4m3 cache, else 1
    int batch, q_len, Hq, Hkv, grp, rows;  // rows = q_len * grp: query rows of a KV head
    int num_blocks, page, max_blocks;
    int window, sinks;
    int scale_block, scale_groups;  // tokens per scale, scales per page
    int box_tok;                    // tokens of one copied box (divides the page and a warp's tile)
    int rb, rbn;                    // row blocks per request; rows of a (full) row block, up to kWinMaxRows
    int ts, tt_log;                 // warps that share a KV head; log2 of a tile's tokens (all of them)
    FastDiv page_div, scale_div, grp_div, rb_div;
    int units;                      // 0: one unit per virtual request, else the balanced unit count
    int nslots;                     // slots of a warp's ring
    bool alone;                     // no more blocks than multiprocessors: each may take one's shared memory
    int withhold;  // test hook of the bounded waits: this unit copies nothing (-1 in every product call)
};

// The tiles of one virtual request.
struct WinVis {
    int n;                // length of the request
    int p_first, p_last;  // positions of the row block's first and last query token
    int lo, hi;           // the windowed run of keys
    int ns, w0;           // sink tiles; first tile of the run after them
    int nt;               // tiles in all
    __device__ __forceinline__ int tile(int j) const { return j < ns ? j : w0 + j - ns; }
};

__device__ __forceinline__ int win_len(const WinArgs& a, int b, int* status) {
    const int n = __ldg(a.seq_lens + b);
    const long long cap = static_cast<long long>(a.max_blocks) * a.page;
    if (n < 0 || n > cap) {
        report(status, MQA_ERR_DEVICE_CHECK);
        return n < 0 ? 0 : static_cast<int>(cap);
    }
    return n;
}

__device__ __forceinline__ WinVis win_visible(const WinArgs& a, int r, int n) {
    WinVis v;
    const int r0 = r * a.rbn, r1 = min(a.rows, r0 + a.rbn) - 1;
    const int i0 = a.q_len == 1 ? 0 : a.grp_div(r0), i1 = a.q_len == 1 ? 0 : a.grp_div(r1);
    const int tl = a.tt_log, up = (1 << tl) - 1;
    v.n = n;
    v.p_first = n - a.q_len + i0;
    v.p_last = n - a.q_len + i1;
    v.hi = max(0, v.p_last + 1);
    v.lo = max(0, v.p_first - a.window + 1);
    const int s_end = min(a.sinks, v.hi);
    v.ns = (s_end + up) >> tl;
    v.w0 = max(v.lo >> tl, v.ns);
    v.nt = v.ns + max(0, ((v.hi + up) >> tl) - v.w0);
    return v;
}

// Balanced mode with T tiles, the longest request's being `longest`: units
// actually used; 0 where a unit is a request.  Where the units are enough for
// the requests and none is much longer than an equal share, cutting would
// cost more, in starts and partials, than it evens out: 256 windows of 128 (512,
// 1024) tokens over int8, 64/8 heads x 64, take 18 (38, 62) us whole and 24
// (43, 63) us cut on 304 units.
__device__ __forceinline__ int win_units(const WinArgs& a, int vb, int T, int longest) {
    const int U = min(a.units, max(1, T)), share = T / U;
    return vb <= a.units && longest <= share + max(2, share / 4) ? 0 : U;
}

// First tile of unit g of U: shares of T / U tiles, the first T % U of them one
// more.  (Moving a cut to a request's boundary where one lies a tile away
// changes nothing: 50.6 and 50.7 us on 64 windows of 1024 over bf16.)
__device__ __forceinline__ int win_unit_start(int T, int U, int g) {
    const int share = T / U;
    return g * share + min(g, T - share * U);
}

// Warps that share a KV head: 8 warps in all, or one per KV head where Hkv
// does not divide 8 evenly.
__host__ __device__ inline int win_subtiles(int hkv) { return hkv == 1 ? 8 : (hkv == 2 ? 4 : (hkv <= 4 ? 2 : 1)); }

// Query rows of a row block at most, and row groups of 8 that they make.  (Four
// groups spill with head size 128: 32 rows take 86 us as one block, 72 as two,
// 16 requests of 4096 tokens, e4m3.)
constexpr int kWinMaxRows = 24;
__host__ __device__ constexpr int win_row_groups(int rbn) { return (rbn + 7) / 8; }

// Thread blocks of stage 1 resident on one SM: one where more than 8 rows meet
// head size 128 (32 windows of 4096, 16 rows, e4m3: 69 us against 92 with two; with
// head size 64 300 windows of 128 with 12 rows take 57 us with one, 39 with two).
__host__ __device__ constexpr int win_ctas_per_sm(int nhb, int D) { return nhb == 1 || (D == 64 && nhb == 2) ? 2 : 1; }
constexpr int kWinMaxCtasPerSm = 2;

// 16-token MMA blocks of a warp's tile, as many as the registers carry beside
// the accumulators.
__host__ __device__ constexpr int win_mblocks(int kind, int nhb, int D) {
    if (nhb == 3) return D == 64 ? 4 : kind == kWinBf16 ? 1 : 2;
    if (D == 64) return kind != kWinBf16 && nhb == 1 ? 4 : 2;
    return kind != kWinBf16 || nhb == 2 ? 2 : 1;
}

cudaError_t win_stage1_bf16(const WinArgs& a, int D, int grid, cudaStream_t stream);
cudaError_t win_stage1_e4m3(const WinArgs& a, int D, int grid, cudaStream_t stream);
cudaError_t win_stage1_int8(const WinArgs& a, int D, int grid, cudaStream_t stream);
cudaError_t win_merge(const WinArgs& a, int D, cudaStream_t stream);

}  // namespace mqa

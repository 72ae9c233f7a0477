// GQA attention of a ragged batch of prompt chunks over a paged cache:
// arguments, the cells and pieces that the work is cut into, and the host
// interface.
//
// A cell is up to 2 * tile_tok consecutive new tokens of one request, for one
// KV head: their query rows (tokens x the grouped heads) fill up to two tiles
// of 128 rows.  Its keys are walked in blocks of 128 tokens (those of the sinks,
// then the run from the first row's window to the last row's limit).  The
// (cell, head) pairs are laid end to end, each with its number of blocks plus
// cell_cost as weight, and cut into one equal share per thread block; what a
// thread block has of one (cell, head) is a piece.  Pieces that hold a whole
// (cell, head) write its result, the others partials that a second kernel
// merges.
#pragma once

#include <cuda.h>

#include "gqa_win.cuh"

namespace mqa {

constexpr int kPreBlock = 128;  // keys of a block
constexpr int kPreTile = 128;   // query rows of a tile
constexpr int kPreMaxBatch = 8192;
constexpr int kPreNoWindow = 1 << 30;

struct PreArgs {
    CUtensorMap q_map;   // {D, Hq, num_tokens}, box {64, grp, tile_tok}
    CUtensorMap kv_map;  // {D, Hkv, rows (block, plane, token)}, box {one line, 1, box_tok}
    const float* kv_scales;  // [blocks, 2, page / scale_block, Hkv], or null
    const float* slopes;     // [Hq], or null
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* query_start;
    const int32_t* prefix_lens;  // [batch], or null
    __nv_bfloat16* out;          // [num_tokens, Hq, D]
    float* lse;                  // [num_tokens, Hq], or null
    // [grid][2], what thread block c leaves for the merge.  Its first piece uses partial slot 2c
    // where it continues a (cell, head) that an earlier block began, its last one slot 2c + 1
    // where it begins one that it does not end.
    //   x  whether the last piece does;  y  the first piece: 0 continues nothing, 1 ends what it
    //   continues, 2 does not, 3 there is no piece at all;  z, w  first row and tokens of the
    //   begun cell;  second x  its KV head
    int4* ws_meta;
    float* ws_ml;                // [2 grid][256][2]: reference (base 2) and sum of each row
    float* ws_o;                 // [2 grid][256][D]
    int* status;
    float sl2;               // scale * log2(e) (times k_scale of a per-tensor e4m3 cache)
    float out_scale;         // v_scale of a per-tensor e4m3 cache, else 1
    float cap2, inv_cap2;    // softcap * log2(e) and its reciprocal, or 0
    float tanh_c[kTanhTerms], tanh_near[kTanhNearTerms];  // cap2 times kTanh and kTanhNear
    float tanh_raw[kTanhNearTerms];             // the latter in products times raw_unit: coefficient k times (sl2 / cap2 / raw_unit)^(2 k + 1)
    float raw_unit;                 // a power of two (1 but over per-tensor e4m3 without slopes)
    bool tiny_unit;                 // .. where these leave the fp32 range, or the cap 2^20
    int num_tokens, batch, Hq, Hkv, grp;
    int tile_tok, tile_rows;  // tokens and rows of a tile: rows = tokens * grp <= 128
    int num_blocks, page, max_blocks;
    int window, sinks;
    int scale_block, scale_groups;
    int box_tok;
    FastDiv page_div, scale_div, grp_div, cell_div;  // cell_div: by 2 * tile_tok
    int cell_cost;  // start and end of a (cell, head), in blocks
    int grid;
    bool cut;  // whether (cell, head) pairs may be cut
    int withhold;  // test hook of the bounded waits: no key of this request is copied (-1 in every product call)
};

// What the cells of a request's tokens see.
struct PreCell {
    int row0;     // first token's row of q and out
    int cnt;      // tokens
    int p0;       // position of the first token
    int n, pre;   // length, bidirectional prefix
    int hi, lo;   // the run of keys that a row of the cell sees: [lo, hi), and the sinks before it
    int s_end;    // end of the sinks
    int ns, w0, nt;  // sink blocks; first block of the run after them; blocks in all
    __device__ __forceinline__ int block(int j) const { return j < ns ? j : w0 + j - ns; }
};

struct PreReq {
    int row0, cnt, n, pre;  // new tokens, length, prefix
};

__device__ __forceinline__ PreReq pre_request(const PreArgs& a, int b, int* status) {
    int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1), n = __ldg(a.seq_lens + b);
    const int cap = a.max_blocks * a.page;
    if (q0 < 0 || q1 < q0 || q1 > a.num_tokens || n < 0 || n > cap) {
        report(status, MQA_ERR_DEVICE_CHECK);
        q0 = min(max(q0, 0), a.num_tokens);
        q1 = min(max(q1, q0), a.num_tokens);
        n = min(max(n, 0), cap);
    }
    PreReq r;
    r.row0 = q0;
    r.cnt = q1 - q0;
    r.n = n;
    r.pre = a.prefix_lens ? min(max(__ldg(a.prefix_lens + b), 0), n) : 0;
    return r;
}

// Cell u of a request.
__device__ __forceinline__ PreCell pre_cell(const PreArgs& a, const PreReq& r, int u) {
    PreCell c;
    const int t0 = u * 2 * a.tile_tok;
    c.row0 = r.row0 + t0;
    c.cnt = min(2 * a.tile_tok, r.cnt - t0);
    c.p0 = r.n - r.cnt + t0;
    c.n = r.n;
    c.pre = r.pre;
    const int last = c.p0 + c.cnt - 1;
    c.hi = last < 0 ? 0 : max(last + 1, r.pre);
    c.lo = max(0, c.p0 - a.window + 1);
    c.s_end = min(a.sinks, c.hi);
    c.ns = (c.s_end + kPreBlock - 1) / kPreBlock;
    c.w0 = max(c.lo / kPreBlock, c.ns);
    c.nt = c.ns + max(0, (c.hi + kPreBlock - 1) / kPreBlock - c.w0);
    return c;
}

// Partials: [2 grid] slots of two tiles.
constexpr int kPreSlotRows = 2 * kPreTile;
inline size_t pre_workspace_bytes(int grid, int D) {
    return static_cast<size_t>(grid) * 2 * sizeof(int4) +
           static_cast<size_t>(grid) * 2 * kPreSlotRows * (D + 2) * sizeof(float);
}

cudaError_t pre_stage1_bf16(const PreArgs& a, int D, cudaStream_t stream);
cudaError_t pre_stage1_e4m3(const PreArgs& a, int D, cudaStream_t stream);
cudaError_t pre_stage1_e4m3_block(const PreArgs& a, int D, cudaStream_t stream);
cudaError_t pre_stage1_int8(const PreArgs& a, int D, cudaStream_t stream);
cudaError_t pre_merge(const PreArgs& a, int D, cudaStream_t stream);

}  // namespace mqa

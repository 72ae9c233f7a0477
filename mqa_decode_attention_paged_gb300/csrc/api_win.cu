// C ABI of windowed and block-scaled GQA decode: argument validation, the
// work split and the launches.  See include/mqa_decode.h for the contract.
#include <cmath>
#include <cstring>

#include "../../include/mqa_decode_testing.h"
#include "api_common.cuh"
#include "gqa_win.cuh"

namespace {

using mqa::api_aligned;
using mqa::api_cuda_fail;

constexpr int kMaxRows = 128;  // query rows of a KV head: q_len * (num_q_heads / num_kv_heads)

struct Rows {
    int grp, rows, rb, rbn;
};

bool heads_ok(int batch, int q_len, int hq, int hkv) {
    return batch >= 1 && q_len >= 1 && hq >= 1 && hkv >= 1 && hq % hkv == 0;
}

bool heads_served(int batch, int q_len, int hq, int hkv) {
    const long long rows = static_cast<long long>(q_len) * (hq / hkv);
    // (the limit on batches counts 16 rows to a block, as the header states it;
    // blocks of 24 rows are fewer, so that the prefix always fits)
    return hkv <= 8 && hq / hkv <= 16 && rows <= kMaxRows &&
           batch <= mqa::kWinMaxVirtual / static_cast<int>((rows + 15) / 16);
}

Rows rows_of(int q_len, int hq, int hkv) {
    Rows r;
    r.grp = hq / hkv;
    r.rows = q_len * r.grp;
    r.rb = (r.rows + mqa::kWinMaxRows - 1) / mqa::kWinMaxRows;
    r.rbn = (r.rows + r.rb - 1) / r.rb;  // (the last block has a row at least)
    return r;
}

// A view of the cache, {line, rows, panels, heads} with rows over blocks,
// planes and tokens, whose box is box_tok rows of one head: it lands as
// [panel][row][line] under the swizzle of its line (128 or 64 bytes).  Encoded
// per call (a fraction of a microsecond): nothing is kept by an address.
bool cache_map(CUtensorMap* out, const void* base, int elt, int D, int hkv, long long rows, int box_tok) {
    auto fn = mqa::api_encode_tiled();
    if (!fn) return false;
    const int line = D * elt >= 128 ? 128 : D * elt;
    const int inner = line / elt, panels = D / inner;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(panels), static_cast<cuuint64_t>(hkv)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(hkv) * D * elt, static_cast<cuuint64_t>(line),
                                   static_cast<cuuint64_t>(D) * elt};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(box_tok),
                               static_cast<cuuint32_t>(panels), 1};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    std::memset(out, 0, sizeof *out);
    return fn(out, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
              const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
              line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether requests are too short to be worth cutting: the window (or the block
// table's width) bounds the bytes of one, which its own block would read in
// `own` us at most, while cutting evens the reading out over the device and
// costs partials and a merge, about 4 us.  One multiprocessor takes in 70 GB/s
// of bf16, 35 GB/s of codes, which it widens; two blocks on it take 2.6 (1.6)
// times as long as one.  Longer windows hold requests of unlike lengths more
// often than not, and are cut (60 us).  Measured whole / cut in us, 32/8 heads x
// 128, bf16, windows of 128, 512 and 1024 tokens: 150 requests 21 / 27, 54 / 61
// and 97 / 104, 200 requests 30 / 33, 95 / 78 and 178 / 135, 304 requests 37 / 44,
// 106 / 110 and 197 / 197 (of 1 to 3000 tokens: 36 / 43, 101 / 101, 179 / 167);
// 64/8 heads x 64, int8, window 128: 100, 150, 200 and 256 requests 13 / 14, 13 /
// 19, 18 / 24, 18 / 24.  These two layouts gave the rates.  Elsewhere (windows
// of 128 and 512): 32/8 x 128, int8, 64 requests 15 / 13 and 36 / 24, 150 17 / 23
// and 37 / 42, 200 24 / 26 and 54 / 51, 304 27 / 35 and 63 / 73; 8/1 x 128, int8,
// 45 requests 9 / 10 and 12 / 11, 150 10 / 14 and 12 / 14; 8/2 x 128, bf16, 45
// requests 9 / 9 and 14 / 12, 150 9 / 13 and 19 / 23.  Of all these the rule takes
// the slower side by more than 5 %, 1 to 5 us, at 128 tokens with 200 requests of
// 8 KV heads x 128 and with 45 of one or two over int8, and at 512 tokens with 150
// requests over codes.
bool whole_requests(const mqa::WinArgs& a, int elt, int head_size, int sms) {
    const long long tt = 1LL << a.tt_log, all = (static_cast<long long>(a.max_blocks) * a.page + tt - 1) / tt;
    const long long seen = (a.sinks + tt - 1) / tt + (static_cast<long long>(a.window) + a.q_len - 2 + tt) / tt + 1;
    const double bytes = static_cast<double>(seen < all ? seen : all) * tt * 2 * a.Hkv * head_size * elt;
    const int vb = a.batch * a.rb;
    const double own = bytes / (elt == 2 ? 70e3 : 35e3), pair = vb <= sms ? 1.0 : elt == 2 ? 2.6 : 1.6;
    return own * pair <= 60.0 && own * pair <= vb * bytes / 6.5e6 + 4.0;
}

mqa_status decode(const void* q, const void* kv_cache, const float* kv_scales, const int32_t* block_table,
                  const int32_t* seq_lens, float scale, float k_scale, float v_scale, int window, int sinks,
                  void* out, float* lse, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_size,
                  int num_blocks, int page_size, int max_blocks, int scale_block, mqa_kv_dtype kv_dtype,
                  int num_kv_splits, void* workspace, size_t workspace_bytes, int* device_status, void* stream,
                  int withhold = -1) {
    // withhold >= 0 only from the test hook mqa_test_gqa_window_withheld
    if (!q || !kv_cache || !block_table || !seq_lens || !out) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(q, 16) || !api_aligned(kv_cache, 16) || !api_aligned(out, 16) || !api_aligned(block_table, 4) ||
        !api_aligned(seq_lens, 4) || (lse && !api_aligned(lse, 4)) ||
        (device_status && !api_aligned(device_status, 4)))
        return MQA_ERR_INVALID_ARG;
    if (!heads_ok(batch, q_len, num_q_heads, num_kv_heads) || num_blocks < 1 || max_blocks < 1 || page_size < 1 ||
        num_kv_splits < 1 || window < 1 || sinks < 0)
        return MQA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return MQA_ERR_INVALID_ARG;
    if (head_size != 64 && head_size != 128) return MQA_ERR_UNSUPPORTED;
    if (!heads_served(batch, q_len, num_q_heads, num_kv_heads)) return MQA_ERR_UNSUPPORTED;
    if (page_size % 16 != 0) return MQA_ERR_UNSUPPORTED;
    const bool block = kv_dtype == MQA_KV_FP8_E4M3_BLOCK || kv_dtype == MQA_KV_INT8_BLOCK;
    if (!block && kv_dtype != MQA_KV_BF16 && kv_dtype != MQA_KV_FP8_E4M3) return MQA_ERR_UNSUPPORTED;
    if (kv_dtype == MQA_KV_FP8_E4M3 && (!std::isfinite(k_scale) || !std::isfinite(v_scale)))
        return MQA_ERR_INVALID_ARG;
    if (block) {
        if (!kv_scales || !api_aligned(kv_scales, 4) || scale_block < 1) return MQA_ERR_INVALID_ARG;
        if (scale_block % 16 != 0 || page_size % scale_block != 0) return MQA_ERR_UNSUPPORTED;
    }
    // positions stay clear of INT_MAX by more than a tile (512 tokens at most),
    // cache rows (two planes of tokens) are ints
    if (static_cast<long long>(max_blocks) * page_size > INT32_MAX - 1024 ||
        static_cast<long long>(num_blocks) * page_size > (1 << 30) - 1)
        return MQA_ERR_UNSUPPORTED;

    const Rows r = rows_of(q_len, num_q_heads, num_kv_heads);
    const int vb = batch * r.rb;
    // the batch's tiles (16 tokens at least, an edge or two more) are counted in ints
    if (vb * ((static_cast<long long>(max_blocks) * page_size >> 4) + 2) > INT32_MAX / 4) return MQA_ERR_UNSUPPORTED;
    const size_t need = gqa_window_decode_workspace_bytes(batch, q_len, num_q_heads, num_kv_heads, head_size,
                                                          num_kv_splits);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MQA_ERR_WORKSPACE_TOO_SMALL;
    if (need > 0 && !api_aligned(workspace, 16)) return MQA_ERR_INVALID_ARG;
    const int sms = mqa::api_sm_count();
    if (sms < 1) return MQA_ERR_CUDA;

    mqa::WinArgs a{};
    const int elt = kv_dtype == MQA_KV_BF16 ? 2 : 1;
    const mqa::WinKind kind = kv_dtype == MQA_KV_BF16         ? mqa::kWinBf16
                              : kv_dtype == MQA_KV_INT8_BLOCK ? mqa::kWinInt8
                                                              : mqa::kWinE4m3;
    const int nhb = mqa::win_row_groups(r.rbn);
    const int warp_tok = 16 * mqa::win_mblocks(kind, nhb, head_size);
    a.ts = mqa::win_subtiles(num_kv_heads);
    a.tt_log = 0;
    while ((1 << a.tt_log) < warp_tok * a.ts) ++a.tt_log;  // (both are powers of two)
    a.page_div = mqa::FastDiv::of(page_size);
    a.scale_div = mqa::FastDiv::of(block ? scale_block : 1);
    a.grp_div = mqa::FastDiv::of(r.grp);
    a.rb_div = mqa::FastDiv::of(r.rb);
    a.box_tok = head_size * elt > 128 ? 16 : warp_tok;  // two panels: a box is an MMA block
    while (page_size % a.box_tok != 0) a.box_tok /= 2;  // a box lies in one page
    if (!cache_map(&a.tmap, kv_cache, elt, head_size, num_kv_heads,
                   2LL * num_blocks * page_size, a.box_tok))
        return api_cuda_fail(cudaErrorInvalidValue);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.kv_scales = block ? kv_scales : nullptr;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.status = device_status;
    const bool per_tensor = kv_dtype == MQA_KV_FP8_E4M3;
    a.sl2 = scale * (per_tensor ? k_scale : 1.0f) * mqa::kLog2e;
    a.out_scale = per_tensor ? v_scale : 1.0f;
    a.batch = batch;
    a.q_len = q_len;
    a.Hq = num_q_heads;
    a.Hkv = num_kv_heads;
    a.grp = r.grp;
    a.rows = r.rows;
    a.rb = r.rb;
    a.rbn = r.rbn;
    a.num_blocks = num_blocks;
    a.page = page_size;
    a.max_blocks = max_blocks;
    a.window = window < mqa::kWinNoWindow ? window : mqa::kWinUnbounded;
    a.sinks = sinks;
    a.withhold = withhold;
    a.scale_block = block ? scale_block : 1;
    a.scale_groups = block ? page_size / scale_block : 1;
    if (num_kv_splits > 1) {
        const size_t slots = static_cast<size_t>(vb) * num_kv_splits;
        a.ws_o = static_cast<float*>(workspace);
        a.ws_lse = a.ws_o + slots * num_kv_heads * r.rbn * head_size;
        a.ws_units = reinterpret_cast<int2*>(a.ws_lse + (slots * num_kv_heads * r.rbn + 1) / 2 * 2);
        // unit g and virtual request v use slot g + v <= units + vb - 2
        const long long cap = static_cast<long long>(vb) * (num_kv_splits - 1) + 1;
        const long long fill = static_cast<long long>(sms) * mqa::win_ctas_per_sm(nhb, head_size);
        // One unit per multiprocessor over bf16 (a block then has a ring of four
        // slots; one request of 8000 or 60000 tokens, 32/8 heads x 128: 13 and 45
        // us, with two units 17 and 55), and over codes where two would leave more
        // than 100 partials a row (one request of 8000, 64/8 heads: 13, 19 us).
        const long long units = kind == mqa::kWinBf16 || fill > 100LL * vb ? sms : fill;
        a.units = static_cast<int>(units < cap ? units : cap);
        if (vb <= fill && whole_requests(a, elt, head_size, sms)) a.units = 0;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int grid = a.units > 0 ? a.units : vb;
    a.alone = grid <= sms;
    const cudaError_t e = kind == mqa::kWinBf16   ? mqa::win_stage1_bf16(a, head_size, grid, st)
                          : kind == mqa::kWinInt8 ? mqa::win_stage1_int8(a, head_size, grid, st)
                                                  : mqa::win_stage1_e4m3(a, head_size, grid, st);
    if (e != cudaSuccess) return api_cuda_fail(e);
    if (a.units > 0)
        if (cudaError_t e2 = mqa::win_merge(a, head_size, st); e2 != cudaSuccess) return api_cuda_fail(e2);
    return MQA_OK;
}

}  // namespace

extern "C" {

size_t gqa_window_decode_workspace_bytes(int batch, int q_len, int num_q_heads, int num_kv_heads, int head_size,
                                         int num_kv_splits) {
    if (!heads_ok(batch, q_len, num_q_heads, num_kv_heads) || head_size < 1 || num_kv_splits < 2) return 0;
    if (!heads_served(batch, q_len, num_q_heads, num_kv_heads)) return 0;
    const Rows r = rows_of(q_len, num_q_heads, num_kv_heads);
    // partials [slots, heads, rows] of head_size + 1 floats (padded to 8
    // bytes), then two ints per virtual request
    const size_t vb = static_cast<size_t>(batch) * r.rb;
    const size_t rows = vb * num_kv_splits * num_kv_heads * r.rbn;
    return rows * head_size * 4 + (rows + 1) / 2 * 8 + vb * 8;
}

int gqa_window_num_kv_splits(int batch, int q_len, int num_q_heads, int num_kv_heads) {
    if (!heads_ok(batch, q_len, num_q_heads, num_kv_heads) ||
        !heads_served(batch, q_len, num_q_heads, num_kv_heads))
        return -1;
    const int sms = mqa::api_sm_count();
    if (sms < 1) return -1;
    const Rows r = rows_of(q_len, num_q_heads, num_kv_heads);
    const int vb = batch * r.rb, fill = sms * mqa::kWinMaxCtasPerSm;
    return 1 + (fill - 1 + vb - 1) / vb;  // the smallest budget that lets units fill the device (2 at least)
}

mqa_status gqa_window_decode(const void* q, const void* kv_cache, const float* kv_scales, const int32_t* block_table,
                             const int32_t* seq_lens, float scale, float k_scale, float v_scale, int window,
                             int sinks, void* out, float* lse, int batch, int q_len, int num_q_heads,
                             int num_kv_heads, int head_size, int num_blocks, int page_size, int max_blocks,
                             int scale_block, mqa_kv_dtype kv_dtype, int num_kv_splits, void* workspace,
                             size_t workspace_bytes, int* device_status, void* stream) {
    return decode(q, kv_cache, kv_scales, block_table, seq_lens, scale, k_scale, v_scale, window, sinks, out, lse,
                  batch, q_len, num_q_heads, num_kv_heads, head_size, num_blocks, page_size, max_blocks, scale_block,
                  kv_dtype, num_kv_splits, workspace, workspace_bytes, device_status, stream);
}

mqa_status gqa_block_decode(const void* q, const void* kv_cache, const float* kv_scales, const int32_t* block_table,
                            const int32_t* seq_lens, float scale, void* out, float* lse, int batch, int q_len,
                            int num_q_heads, int num_kv_heads, int head_size, int num_blocks, int page_size,
                            int max_blocks, int scale_block, mqa_kv_dtype kv_dtype, int num_kv_splits,
                            void* workspace, size_t workspace_bytes, int* device_status, void* stream) {
    if (kv_dtype != MQA_KV_FP8_E4M3_BLOCK && kv_dtype != MQA_KV_INT8_BLOCK) return MQA_ERR_UNSUPPORTED;
    return decode(q, kv_cache, kv_scales, block_table, seq_lens, scale, 1.0f, 1.0f, mqa::kWinNoWindow, 0, out, lse,
                  batch, q_len, num_q_heads, num_kv_heads, head_size, num_blocks, page_size, max_blocks, scale_block,
                  kv_dtype, num_kv_splits, workspace, workspace_bytes, device_status, stream);
}

mqa_status mqa_test_gqa_window_withheld(const void* q, const void* kv_cache, const float* kv_scales,
                                        const int32_t* block_table, const int32_t* seq_lens, float scale, int window,
                                        int sinks, void* out, float* lse, int batch, int q_len, int num_q_heads,
                                        int num_kv_heads, int head_size, int num_blocks, int page_size,
                                        int max_blocks, int scale_block, mqa_kv_dtype kv_dtype, int num_kv_splits,
                                        void* workspace, size_t workspace_bytes, int* device_status, void* stream,
                                        int withhold_unit) {
    if (!mqa::api_test_hooks()) return MQA_ERR_UNSUPPORTED;
    if (withhold_unit < 0) return MQA_ERR_INVALID_ARG;
    return decode(q, kv_cache, kv_scales, block_table, seq_lens, scale, 1.0f, 1.0f, window, sinks, out, lse, batch,
                  q_len, num_q_heads, num_kv_heads, head_size, num_blocks, page_size, max_blocks, scale_block,
                  kv_dtype, num_kv_splits, workspace, workspace_bytes, device_status, stream, withhold_unit);
}

}  // extern "C"

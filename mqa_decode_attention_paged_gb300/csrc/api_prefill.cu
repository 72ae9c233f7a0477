// C ABI of prompt attention over paged GQA caches: argument validation and the
// launches.  See include/mqa_decode.h for the contract.
#include <cmath>
#include <cstring>

#include "../../include/mqa_decode_testing.h"
#include "api_common.cuh"
#include "gqa_prefill.cuh"

namespace {

using mqa::api_aligned;
using mqa::api_cuda_fail;
using mqa::ApiSpan;

constexpr int kMaxGrid = 256;  // thread blocks that the merge looks over
constexpr int kMaxTokens = 1 << 24;

bool heads_ok(int hq, int hkv) { return hq >= 1 && hkv >= 1 && hq % hkv == 0; }
bool heads_served(int hq, int hkv) { return hkv <= 128 && hq / hkv <= 128; }

int grid_of() {
    const int sms = mqa::api_sm_count();
    return sms < kMaxGrid ? sms : kMaxGrid;
}

bool encode3(CUtensorMap* out, const void* base, int elt, long long d0, long long d1, long long d2, long long s1,
             long long s2, int b0, int b1, int b2) {
    auto fn = mqa::api_encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(s2)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(b0), static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
    const cuuint32_t step[3] = {1, 1, 1};
    std::memset(out, 0, sizeof *out);
    return fn(out, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
              const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              b0 * elt == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

mqa_status prefill(const void* q, const void* kv_cache, const float* kv_scales, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* query_start, const int32_t* prefix_lens, float scale,
                   float k_scale, float v_scale, float softcap, const float* slopes, int window, int sinks, void* out,
                   float* lse, int num_tokens, int batch, int num_q_heads, int num_kv_heads, int head_size,
                   int num_blocks, int page_size, int max_blocks, int scale_block, mqa_kv_dtype kv_dtype,
                   long long q_stride, int num_kv_splits, void* workspace, size_t workspace_bytes, int* device_status,
                   void* stream, int withhold = -1) {
    // withhold >= 0 only from the test hook mqa_test_gqa_prefill_withheld
    if (!kv_cache || !block_table || !seq_lens || !query_start || num_tokens < 0) return MQA_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!q || !out)) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(q, 16) || !api_aligned(kv_cache, 16) || !api_aligned(out, 16) || !api_aligned(block_table, 4) ||
        !api_aligned(seq_lens, 4) || !api_aligned(query_start, 4) || !api_aligned(prefix_lens, 4) ||
        !api_aligned(slopes, 4) || !api_aligned(lse, 4) || !api_aligned(device_status, 4))
        return MQA_ERR_INVALID_ARG;
    if (batch < 1 || !heads_ok(num_q_heads, num_kv_heads) || num_blocks < 1 || max_blocks < 1 || page_size < 1 ||
        num_kv_splits < 1 || window < 1 || sinks < 0)
        return MQA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !mqa::api_softcap_ok(softcap)) return MQA_ERR_INVALID_ARG;
    if (head_size != 64 && head_size != 128) return MQA_ERR_UNSUPPORTED;
    if (!heads_served(num_q_heads, num_kv_heads) || page_size % 16 != 0) return MQA_ERR_UNSUPPORTED;
    if (num_tokens > kMaxTokens || batch > mqa::kPreMaxBatch) return MQA_ERR_UNSUPPORTED;
    const bool block = kv_dtype == MQA_KV_FP8_E4M3_BLOCK || kv_dtype == MQA_KV_INT8_BLOCK;
    if (!block && kv_dtype != MQA_KV_BF16 && kv_dtype != MQA_KV_FP8_E4M3) return MQA_ERR_UNSUPPORTED;
    if (kv_dtype == MQA_KV_FP8_E4M3 && (!std::isfinite(k_scale) || !std::isfinite(v_scale))) return MQA_ERR_INVALID_ARG;
    if (block) {
        if (!kv_scales || !api_aligned(kv_scales, 4) || scale_block < 1) return MQA_ERR_INVALID_ARG;
        if (scale_block % 16 != 0 || page_size % scale_block != 0) return MQA_ERR_UNSUPPORTED;
    }
    // positions (less a window of 2^30) and cache rows (two planes) are ints
    if (static_cast<long long>(max_blocks) * page_size > (1 << 30) - 1 ||
        static_cast<long long>(num_blocks) * page_size > (1 << 30) - 1)
        return MQA_ERR_UNSUPPORTED;
    // a token's row of q: dense, 16-byte aligned
    if (q_stride % 8 != 0 || q_stride < static_cast<long long>(num_q_heads) * head_size || q_stride > (1LL << 36))
        return MQA_ERR_INVALID_ARG;
    if (num_kv_splits > 1 && !workspace) return MQA_ERR_WORKSPACE_TOO_SMALL;
    // (rows of q and the rest are read while others' results are written)
    const size_t q_bytes = num_tokens > 0 ? 2 * ((num_tokens - 1) * static_cast<size_t>(q_stride) + static_cast<size_t>(num_q_heads) * head_size) : 0;
    const size_t rows = static_cast<size_t>(num_tokens) * num_q_heads;
    const size_t lines = 2ull * num_blocks * page_size * num_kv_heads;  // rows of head_size codes of the cache
    const ApiSpan writes[] = {{out, rows * head_size * 2}, {lse, rows * 4}, {device_status, 4},
                              {num_kv_splits > 1 ? workspace : nullptr, workspace_bytes}};
    const ApiSpan reads[] = {{q, q_bytes}, {kv_cache, lines * head_size * (kv_dtype == MQA_KV_BF16 ? 2 : 1)},
                             {block ? kv_scales : nullptr, block ? lines / scale_block * 4 : 0},
                             {block_table, static_cast<size_t>(batch) * max_blocks * 4}, {seq_lens, batch * 4ull},
                             {query_start, (batch + 1) * 4ull}, {prefix_lens, batch * 4ull}, {slopes, num_q_heads * 4ull}};
    if (mqa::api_clash(writes, reads)) return MQA_ERR_INVALID_ARG;
    const int grid = grid_of();
    if (grid < 1) return MQA_ERR_CUDA;
    const size_t need = num_kv_splits > 1 ? mqa::pre_workspace_bytes(grid, head_size) : 0;
    if (need > 0 && workspace_bytes < need) return MQA_ERR_WORKSPACE_TOO_SMALL;
    if (need > 0 && !api_aligned(workspace, 16)) return MQA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MQA_OK;

    mqa::PreArgs a{};
    const int elt = kv_dtype == MQA_KV_BF16 ? 2 : 1;
    a.grp = num_q_heads / num_kv_heads;
    a.tile_tok = mqa::kPreTile / a.grp;
    a.tile_rows = a.tile_tok * a.grp;
    a.box_tok = mqa::kPreBlock;
    while (page_size % a.box_tok != 0) a.box_tok /= 2;  // a box lies in one page
    const int line = head_size * elt >= 128 ? 128 / elt : head_size;  // columns of one swizzled line
    if (!encode3(&a.q_map, q, 2, head_size, num_q_heads, num_tokens, head_size * 2LL, q_stride * 2, 64, a.grp, a.tile_tok) ||
        !encode3(&a.kv_map, kv_cache, elt, head_size, num_kv_heads, 2LL * num_blocks * page_size,
                 static_cast<long long>(head_size) * elt, static_cast<long long>(num_kv_heads) * head_size * elt, line, 1,
                 a.box_tok))
        return api_cuda_fail(cudaErrorInvalidValue);
    a.kv_scales = block ? kv_scales : nullptr;
    a.slopes = slopes;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.query_start = query_start;
    a.prefix_lens = prefix_lens;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.status = device_status;
    const bool per_tensor = kv_dtype == MQA_KV_FP8_E4M3;
    a.sl2 = scale * (per_tensor ? k_scale : 1.f) * mqa::kLog2e;
    a.out_scale = per_tensor ? v_scale : 1.f;
    a.cap2 = softcap * mqa::kLog2e;
    for (int k = 0; k < mqa::kTanhTerms; ++k) a.tanh_c[k] = a.cap2 * mqa::kTanh[k];
    for (int k = 0; k < mqa::kTanhNearTerms; ++k) a.tanh_near[k] = a.cap2 * mqa::kTanhNear[k];
    a.inv_cap2 = softcap > 0.f ? 1.f / a.cap2 : 0.f;
    a.num_tokens = num_tokens;
    a.batch = batch;
    a.Hq = num_q_heads;
    a.Hkv = num_kv_heads;
    a.num_blocks = num_blocks;
    a.page = page_size;
    a.max_blocks = max_blocks;
    a.window = window < mqa::kPreNoWindow ? window : mqa::kPreNoWindow;
    a.sinks = sinks;
    a.scale_block = block ? scale_block : 1;
    a.scale_groups = block ? page_size / scale_block : 1;
    a.page_div = mqa::FastDiv::of(page_size);
    a.scale_div = mqa::FastDiv::of(a.scale_block);
    a.grp_div = mqa::FastDiv::of(a.grp);
    a.cell_div = mqa::FastDiv::of(2 * a.tile_tok);
    // What a (cell, head) takes beside its blocks (Q's copy, the first product, the
    // output), in blocks: with 1, 2, 3 and 4 one prompt of 15999 tokens takes 1740,
    // 1526, 1385 and 1383 us, six of 500 to 2600 202, 170, 165 and 171; capped, where
    // a block takes longer, 2 and 3 are within 2 % of each other.
    a.cell_cost = 3;
    const double unit = softcap > 0.f ? static_cast<double>(a.sl2) * a.inv_cap2 : 0.0;
    auto coefficients = [&](double of) {
        double power = of;
        for (int k = 0; k < mqa::kTanhNearTerms; ++k, power *= of * of) a.tanh_raw[k] = static_cast<float>(a.cap2 * mqa::kTanhNear[k] * power);
        // normal numbers (full precision, and infinite times a masked key's infinity)
        return std::fabs(a.tanh_raw[mqa::kTanhNearTerms - 1]) >= 0x1p-126f;
    };
    // Over per-tensor e4m3 k_scale is part of the unit (cap 50, head size 128: k_scales below 0.035): small units leave a power of
    // two to the products there.  One prompt of 15999 tokens, cap 50: 2600 us, with k_scale 0.02 2536, in the slow form 8450.
    // (With the same multiplication bf16 takes 2077 instead of 1854, and e4m3 with slopes too 4151 instead of 3784.)
    a.raw_unit = 1.f;
    bool fit = coefficients(unit);
    if (!fit && per_tensor && !slopes && std::fabs(unit) >= 0x1p-60) {
        a.raw_unit = static_cast<float>(std::ldexp(1.0, std::ilogb(unit)));
        fit = coefficients(unit / a.raw_unit);
    }
    // The slow form for every block where they do not fit.  Logits beyond 2^20 are taken relative to the largest of the same
    // capped values, not to the cap of the largest product, whose rounding they may exceed by more than an exponential
    // holds.
    a.tiny_unit = std::fabs(unit) > 1.0 || !fit || a.cap2 > 0x1p20f;
    a.grid = grid;
    a.cut = num_kv_splits > 1;
    a.withhold = withhold;
    if (a.cut) {
        a.ws_meta = static_cast<int4*>(workspace);
        a.ws_ml = reinterpret_cast<float*>(a.ws_meta + 2 * grid);
        a.ws_o = a.ws_ml + 2LL * grid * mqa::kPreSlotRows * 2;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_dtype == MQA_KV_BF16        ? mqa::pre_stage1_bf16(a, head_size, st)
                          : kv_dtype == MQA_KV_INT8_BLOCK ? mqa::pre_stage1_int8(a, head_size, st)
                          : block                         ? mqa::pre_stage1_e4m3_block(a, head_size, st)
                                                          : mqa::pre_stage1_e4m3(a, head_size, st);
    if (e != cudaSuccess) return api_cuda_fail(e);
    if (a.cut)
        if (cudaError_t e2 = mqa::pre_merge(a, head_size, st); e2 != cudaSuccess) return api_cuda_fail(e2);
    return MQA_OK;
}

}  // namespace

extern "C" {

size_t gqa_prefill_workspace_bytes(int num_q_heads, int num_kv_heads, int head_size) {
    if (!heads_ok(num_q_heads, num_kv_heads) || !heads_served(num_q_heads, num_kv_heads)) return 0;
    if (head_size != 64 && head_size != 128) return 0;
    const int grid = grid_of();
    return grid < 1 ? 0 : mqa::pre_workspace_bytes(grid, head_size);
}

mqa_status gqa_prefill(const void* q, const void* kv_cache, const float* kv_scales, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* query_start, const int32_t* prefix_lens, float scale,
                       float k_scale, float v_scale, float softcap, const float* slopes, int window, int sinks,
                       void* out, float* lse, int num_tokens, int batch, int num_q_heads, int num_kv_heads,
                       int head_size, int num_blocks, int page_size, int max_blocks, int scale_block,
                       mqa_kv_dtype kv_dtype, long long q_stride, int num_kv_splits, void* workspace,
                       size_t workspace_bytes, int* device_status, void* stream) {
    return prefill(q, kv_cache, kv_scales, block_table, seq_lens, query_start, prefix_lens, scale, k_scale, v_scale,
                   softcap, slopes, window, sinks, out, lse, num_tokens, batch, num_q_heads, num_kv_heads, head_size,
                   num_blocks, page_size, max_blocks, scale_block, kv_dtype, q_stride, num_kv_splits, workspace,
                   workspace_bytes, device_status, stream);
}

mqa_status mqa_test_gqa_prefill_withheld(const void* q, const void* kv_cache, const int32_t* block_table,
                                         const int32_t* seq_lens, const int32_t* query_start, float scale, void* out,
                                         int num_tokens, int batch, int num_q_heads, int num_kv_heads, int head_size,
                                         int num_blocks, int page_size, int max_blocks, long long q_stride,
                                         int* device_status, void* stream, int withhold_request) {
    if (!mqa::api_test_hooks()) return MQA_ERR_UNSUPPORTED;
    if (withhold_request < 0) return MQA_ERR_INVALID_ARG;
    return prefill(q, kv_cache, nullptr, block_table, seq_lens, query_start, nullptr, scale, 1.f, 1.f, 0.f, nullptr,
                   mqa::kPreNoWindow, 0, out, nullptr, num_tokens, batch, num_q_heads, num_kv_heads, head_size,
                   num_blocks, page_size, max_blocks, 0, MQA_KV_BF16, q_stride, 1, nullptr, 0, device_status, stream,
                   withhold_request);
}

}  // extern "C"

// C ABI of the cache-append entry points: argument validation and launches.
// See include/mqa_decode.h for the contract.
#include <cmath>

#include "api_common.cuh"
#include "append.cuh"

namespace {

using mqa::api_aligned;

// Row strides are multiples of 8 elements (16-byte loads) and hold a row.
bool stride_ok(long long s, long long least) { return s >= least && s % 8 == 0; }

// A per-tensor scale that can be divided by: its reciprocal is a normal number.
bool scale_ok(float s) { return std::fabs(s) >= 0x1p-126f && std::fabs(s) <= 0x1p126f; }

// The checks the two entry points share; MQA_OK if the call may go on.
mqa_status check_batch(const mqa::AppendBatch& t) {
    if (!t.cos_sin || !t.block_table || !t.seq_lens || !t.query_start) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(t.cos_sin, 16) || !api_aligned(t.block_table, 4) || !api_aligned(t.seq_lens, 4) ||
        !api_aligned(t.query_start, 4) || (t.status && !api_aligned(t.status, 4)))
        return MQA_ERR_INVALID_ARG;
    if (t.tokens < 0 || t.batch < 1 || t.num_blocks < 1 || t.page < 1 || t.max_blocks < 1 || t.max_position < 1 ||
        t.rotary < 1)
        return MQA_ERR_INVALID_ARG;
    if (t.page % 16 != 0 || t.rotary % 16 != 0 || t.batch > (1 << 20) || t.tokens > (1 << 24))
        return MQA_ERR_UNSUPPORTED;
    if (static_cast<long long>(t.max_blocks) * t.page > INT32_MAX ||
        static_cast<long long>(t.num_blocks) * t.page > INT32_MAX)
        return MQA_ERR_UNSUPPORTED;
    return MQA_OK;
}

}  // namespace

extern "C" {

mqa_status gqa_rope_append(const void* q, const void* k, const void* v, const float* cos_sin,
                           const int32_t* query_start, const int32_t* seq_lens, const int32_t* block_table,
                           void* q_out, void* kv_cache, float* kv_scales, float k_scale, float v_scale,
                           int num_tokens, int batch, int num_q_heads, int num_kv_heads, int head_size,
                           int rotary_dim, int interleaved, int max_position, int num_blocks, int page_size,
                           int max_blocks, int scale_block, mqa_kv_dtype kv_dtype, long long q_stride,
                           long long k_stride, long long v_stride, long long q_out_stride, int* device_status,
                           void* stream) {
    mqa::GqaAppendArgs a{};
    a.t = {cos_sin,    block_table,      seq_lens,     query_start, device_status, num_tokens, batch,
           rotary_dim, interleaved != 0, max_position, num_blocks,  page_size,     max_blocks};
    if (!k || !v || !kv_cache || (q != nullptr) != (q_out != nullptr)) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(k, 16) || !api_aligned(v, 16) || !api_aligned(kv_cache, 16) || !api_aligned(q, 16) ||
        !api_aligned(q_out, 16))
        return MQA_ERR_INVALID_ARG;
    if (num_kv_heads < 1 || (q && num_q_heads < 1)) return MQA_ERR_INVALID_ARG;
    if (const mqa_status s = check_batch(a.t); s != MQA_OK) return s;
    if (head_size != 64 && head_size != 128) return MQA_ERR_UNSUPPORTED;
    if (rotary_dim > head_size) return MQA_ERR_INVALID_ARG;
    if (num_kv_heads > 8 || num_q_heads > 1024) return MQA_ERR_UNSUPPORTED;
    if (kv_dtype < MQA_KV_BF16 || kv_dtype > MQA_KV_INT8_BLOCK) return MQA_ERR_UNSUPPORTED;
    const long long kv_row = static_cast<long long>(num_kv_heads) * head_size;
    if (!stride_ok(k_stride, kv_row) || !stride_ok(v_stride, kv_row)) return MQA_ERR_INVALID_ARG;
    if (q) {
        const long long q_row = static_cast<long long>(num_q_heads) * head_size;
        if (!stride_ok(q_stride, q_row) || !stride_ok(q_out_stride, q_row)) return MQA_ERR_INVALID_ARG;
    }
    if (kv_dtype == MQA_KV_FP8_E4M3 && (!scale_ok(k_scale) || !scale_ok(v_scale))) return MQA_ERR_INVALID_ARG;
    if (kv_dtype == MQA_KV_FP8_E4M3_BLOCK || kv_dtype == MQA_KV_INT8_BLOCK) {
        if (!kv_scales || !api_aligned(kv_scales, 4) || scale_block < 1) return MQA_ERR_INVALID_ARG;
        if (scale_block % 16 != 0 || page_size % scale_block != 0) return MQA_ERR_UNSUPPORTED;
    }
    if (num_tokens == 0) return MQA_OK;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.q_out = static_cast<__nv_bfloat16*>(q_out);
    a.cache = static_cast<uint8_t*>(kv_cache);
    a.scales = kv_scales;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qo_stride = q_out_stride;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.Hq = q ? num_q_heads : 0;
    a.Hkv = num_kv_heads;
    a.scale_block = scale_block;
    const cudaError_t e = mqa::gqa_append(a, head_size, static_cast<int>(kv_dtype), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MQA_OK : mqa::api_cuda_fail(e);
}

mqa_status mla_rope_append(const void* kv_c, const void* k_pe, const void* q_pe, const float* cos_sin,
                           const int32_t* query_start, const int32_t* seq_lens, const int32_t* block_table,
                           void* q_pe_out, void* kv_cache, float k_scale, int num_tokens, int batch, int num_heads,
                           int head_size, int kv_lora_rank, int interleaved, int max_position, int num_blocks,
                           int page_size, int max_blocks, mqa_kv_dtype kv_dtype, long long kv_c_stride,
                           long long k_pe_stride, long long q_pe_stride, long long q_pe_head_stride,
                           long long q_out_stride, long long q_out_head_stride, int* device_status, void* stream) {
    mqa::MlaAppendArgs a{};
    a.t = {cos_sin, block_table,      seq_lens,     query_start, device_status, num_tokens, batch,
           64,      interleaved != 0, max_position, num_blocks,  page_size,     max_blocks};
    if (!kv_c || !k_pe || !kv_cache || (q_pe != nullptr) != (q_pe_out != nullptr)) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(kv_c, 16) || !api_aligned(k_pe, 16) || !api_aligned(kv_cache, 16) || !api_aligned(q_pe, 16) ||
        !api_aligned(q_pe_out, 16))
        return MQA_ERR_INVALID_ARG;
    if (q_pe && num_heads < 1) return MQA_ERR_INVALID_ARG;
    if (const mqa_status s = check_batch(a.t); s != MQA_OK) return s;
    if (!((head_size == 576 && kv_lora_rank == 512) || (head_size == 320 && kv_lora_rank == 256)))
        return MQA_ERR_UNSUPPORTED;
    if (num_heads > 1024) return MQA_ERR_UNSUPPORTED;
    if (kv_dtype != MQA_KV_BF16 && kv_dtype != MQA_KV_FP8_E4M3) return MQA_ERR_UNSUPPORTED;
    if (!stride_ok(kv_c_stride, kv_lora_rank) || !stride_ok(k_pe_stride, 64)) return MQA_ERR_INVALID_ARG;
    if (q_pe && (!stride_ok(q_pe_head_stride, 64) || !stride_ok(q_out_head_stride, 64) ||
                 !stride_ok(q_pe_stride, 64) || !stride_ok(q_out_stride, 64)))
        return MQA_ERR_INVALID_ARG;
    // rows that are written lie apart: a token's heads within its stride, or a head's tokens within the head's
    if (q_pe && q_out_stride < (num_heads - 1) * q_out_head_stride + 64 &&
        q_out_head_stride < (num_tokens - 1) * q_out_stride + 64)
        return MQA_ERR_INVALID_ARG;
    if (kv_dtype == MQA_KV_FP8_E4M3 && !scale_ok(k_scale)) return MQA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MQA_OK;
    a.kv_c = static_cast<const __nv_bfloat16*>(kv_c);
    a.k_pe = static_cast<const __nv_bfloat16*>(k_pe);
    a.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
    a.q_out = static_cast<__nv_bfloat16*>(q_pe_out);
    a.cache = static_cast<uint8_t*>(kv_cache);
    a.c_stride = kv_c_stride;
    a.p_stride = k_pe_stride;
    a.q_stride = q_pe_stride;
    a.qh_stride = q_pe_head_stride;
    a.qo_stride = q_out_stride;
    a.qoh_stride = q_out_head_stride;
    a.k_scale = k_scale;
    a.H = q_pe ? num_heads : 0;
    a.R = kv_lora_rank;
    const cudaError_t e = mqa::mla_append(a, kv_dtype == MQA_KV_FP8_E4M3, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MQA_OK : mqa::api_cuda_fail(e);
}

}  // extern "C"

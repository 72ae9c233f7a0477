// Appending new tokens to a paged cache with the rotary position applied:
// arguments and host interface (append.cu).
#pragma once

#include "common.cuh"

namespace mqa {

// The ragged batch and where its tokens go.
struct AppendBatch {
    const float* cos_sin;        // [max_position, rotary]: cos | sin
    const int32_t* block_table;  // [batch, max_blocks]
    const int32_t* seq_lens;     // [batch], the new tokens included
    const int32_t* query_start;  // [batch + 1]: request b has tokens [query_start[b], query_start[b + 1])
    int* status;
    int tokens, batch, rotary, interleaved;
    int max_position, num_blocks, page, max_blocks;
};

struct GqaAppendArgs {
    AppendBatch t;
    const __nv_bfloat16 *q, *k, *v;  // token strides below, [heads, D] dense within a token
    __nv_bfloat16* q_out;
    uint8_t* cache;  // [blocks, 2, page, Hkv, row bytes]
    float* scales;   // [blocks, 2, page / scale_block, Hkv] (block formats)
    long long q_stride, k_stride, v_stride, qo_stride;  // elements
    float k_scale, v_scale;  // per-tensor e4m3
    int Hq, Hkv;             // Hq = 0: no query
    int scale_block;
};

struct MlaAppendArgs {
    AppendBatch t;
    const __nv_bfloat16 *kv_c, *k_pe, *q_pe;
    __nv_bfloat16* q_out;
    uint8_t* cache;  // [blocks, page, R + 64]
    long long c_stride, p_stride, q_stride, qh_stride, qo_stride, qoh_stride;  // elements
    float k_scale;
    int H, R;  // H = 0: no query
};

// kv_dtype: a value of mqa_kv_dtype.
cudaError_t gqa_append(const GqaAppendArgs& a, int D, int kv_dtype, cudaStream_t stream);
cudaError_t mla_append(const MlaAppendArgs& a, bool fp8, cudaStream_t stream);

}  // namespace mqa

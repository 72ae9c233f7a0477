// C ABI of the page operations: argument validation and the launches.  See
// include/mqa_decode.h for the contract.
#include <algorithm>
#include <utility>

#include "api_common.cuh"
#include "pages.cuh"

namespace {

using mqa::api_aligned;
using mqa::api_cuda_fail;
using mqa::api_overlap;
using mqa::ApiSpan;

// Where the caches lie, in ascending order.
struct Places {
    std::pair<uintptr_t, uintptr_t> at[mqa::kMaxPools];
    int n;
    // Whether one of them holds bytes of the span.
    bool hold(const ApiSpan& s) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(s.p);
        const auto* e = std::partition_point(at, at + n, [a](const auto& x) { return x.second <= a; });
        return s.p && e != at + n && e->first < a + s.n;
    }
    template <int N>
    bool hold_any(const ApiSpan (&spans)[N]) const {
        return std::any_of(spans, spans + N, [this](const ApiSpan& s) { return hold(s); });
    }
};

// The caches as pools.
mqa_status pools_of(mqa::PagePools& p, Places& where, void* const* caches, const size_t* page_bytes, int n, int num_blocks) {
    if (n < 0 || (n > 0 && (!caches || !page_bytes))) return MQA_ERR_INVALID_ARG;
    if (n > mqa::kMaxPools) return MQA_ERR_UNSUPPORTED;
    long long chunks = 0;
    for (int i = 0; i < n; ++i) {
        if (!caches[i] || !api_aligned(caches[i], 16) || page_bytes[i] < 4) return MQA_ERR_INVALID_ARG;
        if (page_bytes[i] % 4 != 0 || page_bytes[i] > (1ull << 30)) return MQA_ERR_UNSUPPORTED;
        const uintptr_t at = reinterpret_cast<uintptr_t>(caches[i]);
        where.at[i] = {at, at + page_bytes[i] * static_cast<size_t>(num_blocks)};
        p.pool[i].base = static_cast<char*>(caches[i]);
        p.pool[i].bytes = static_cast<long long>(page_bytes[i]);
        p.first[i] = static_cast<int>(chunks);
        chunks += (p.pool[i].bytes + mqa::kPageChunk - 1) / mqa::kPageChunk;
    }
    // (two pools in one place would be copied by two blocks at once)
    std::sort(where.at, where.at + n);
    for (int i = 1; i < n; ++i)
        if (where.at[i].first < where.at[i - 1].second) return MQA_ERR_INVALID_ARG;
    where.n = n;
    p.first[n] = static_cast<int>(chunks);
    p.n = n;
    return MQA_OK;
}

mqa_status sizes_ok(int rows, int new_rows, int max_blocks, int num_blocks, int page_size) {
    if (rows < 1 || new_rows < 1 || max_blocks < 1 || num_blocks < 1 || page_size < 1) return MQA_ERR_INVALID_ARG;
    if (page_size % 16 != 0 || rows > mqa::kPagesMaxRows || new_rows > mqa::kPagesMaxRows || num_blocks > (1 << 30))
        return MQA_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_blocks) * page_size > INT32_MAX - 1024) return MQA_ERR_UNSUPPORTED;
    return MQA_OK;
}

}  // namespace

extern "C" {

size_t mqa_pages_fork_workspace_bytes(int new_rows) {
    return new_rows < 1 || new_rows > mqa::kPagesMaxRows ? 0 : mqa::fork_workspace_bytes(new_rows);
}

size_t mqa_pages_compact_workspace_bytes(int num_blocks) {
    return num_blocks < 1 || num_blocks > (1 << 30) ? 0 : mqa::compact_workspace_bytes(num_blocks);
}

mqa_status mqa_pages_fork(const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                          const int32_t* refs, int32_t* new_table, int32_t* new_lens, int32_t* new_refs, int rows,
                          int new_rows, int max_blocks, int num_blocks, int page_size, void* const* caches,
                          const size_t* page_bytes, int num_caches, void* workspace, size_t workspace_bytes,
                          int* device_status, void* stream) {
    if (!block_table || !seq_lens || !parents || !refs || !new_table || !new_lens || !new_refs) return MQA_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(parents), static_cast<const void*>(refs),
                          static_cast<const void*>(new_table), static_cast<const void*>(new_lens),
                          static_cast<const void*>(new_refs), static_cast<const void*>(device_status)})
        if (!api_aligned(p, 4)) return MQA_ERR_INVALID_ARG;
    if (const mqa_status s = sizes_ok(rows, new_rows, max_blocks, num_blocks, page_size); s != MQA_OK) return s;
    // outputs on the inputs that they follow from; every other pair below, where the workspace is known
    const size_t old_table = static_cast<size_t>(rows) * max_blocks * 4, table = static_cast<size_t>(new_rows) * max_blocks * 4;
    if (api_overlap(block_table, old_table, new_table, table) || api_overlap(seq_lens, rows * 4ull, new_lens, new_rows * 4ull) ||
        (refs != new_refs && api_overlap(refs, num_blocks * 4ull, new_refs, num_blocks * 4ull)))
        return MQA_ERR_INVALID_ARG;
    mqa::PagePools pools;
    Places places;
    if (const mqa_status s = pools_of(pools, places, caches, page_bytes, num_caches, num_blocks); s != MQA_OK) return s;
    if (!workspace || workspace_bytes < mqa::fork_workspace_bytes(new_rows)) return MQA_ERR_WORKSPACE_TOO_SMALL;
    // blocks read what others write
    const size_t row_bytes = new_rows * 4ull, ref_bytes = num_blocks * 4ull;
    const ApiSpan writes[] = {{new_table, table}, {new_lens, row_bytes}, {new_refs, ref_bytes}, {device_status, 4},
                              {workspace, mqa::fork_workspace_bytes(new_rows)}};
    const ApiSpan reads[] = {{block_table, old_table}, {seq_lens, rows * 4ull}, {parents, row_bytes},
                             {refs == new_refs ? nullptr : refs, ref_bytes}};
    if (mqa::api_clash(writes, reads) || places.hold_any(writes) || places.hold_any(reads)) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(workspace, 16)) return MQA_ERR_INVALID_ARG;
    const int sms = mqa::api_sm_count();
    if (sms < 1) return MQA_ERR_CUDA;
    mqa::PagesArgs a{};
    a.table = block_table;
    a.lens = seq_lens;
    a.parents = parents;
    a.refs = refs;
    a.new_table = new_table;
    a.new_lens = new_lens;
    a.new_refs = new_refs;
    a.ws = static_cast<int32_t*>(workspace);
    a.status = device_status;
    a.rows = rows;
    a.new_rows = new_rows;
    a.width = max_blocks;
    a.num_blocks = num_blocks;
    a.page = page_size;
    const cudaError_t e = mqa::pages_fork(a, pools, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MQA_OK : api_cuda_fail(e);
}

mqa_status mqa_pages_compact(const int32_t* block_table, const int32_t* seq_lens, const int32_t* refs,
                             int32_t* new_table, int32_t* new_refs, int32_t* moved, int32_t* num_live, int rows,
                             int max_blocks, int num_blocks, int page_size, void* const* caches,
                             const size_t* page_bytes, int num_caches, void* workspace, size_t workspace_bytes,
                             int* device_status, void* stream) {
    if (!block_table || !seq_lens || !refs || !new_table || !new_refs || !moved || !num_live) return MQA_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(refs), static_cast<const void*>(new_table),
                          static_cast<const void*>(new_refs), static_cast<const void*>(moved),
                          static_cast<const void*>(num_live), static_cast<const void*>(device_status)})
        if (!api_aligned(p, 4)) return MQA_ERR_INVALID_ARG;
    if (const mqa_status s = sizes_ok(rows, rows, max_blocks, num_blocks, page_size); s != MQA_OK) return s;
    const size_t table = static_cast<size_t>(rows) * max_blocks * 4;
    if ((block_table != new_table && api_overlap(block_table, table, new_table, table)) ||
        (refs != new_refs && api_overlap(refs, num_blocks * 4ull, new_refs, num_blocks * 4ull)) ||
        api_overlap(moved, num_blocks * 4ull, refs, num_blocks * 4ull) || api_overlap(moved, num_blocks * 4ull, new_refs, num_blocks * 4ull))
        return MQA_ERR_INVALID_ARG;
    mqa::PagePools pools;
    Places places;
    if (const mqa_status s = pools_of(pools, places, caches, page_bytes, num_caches, num_blocks); s != MQA_OK) return s;
    if (!workspace || workspace_bytes < mqa::compact_workspace_bytes(num_blocks)) return MQA_ERR_WORKSPACE_TOO_SMALL;
    const size_t ref_bytes = num_blocks * 4ull;
    const ApiSpan writes[] = {{new_table, table}, {new_refs, ref_bytes}, {moved, ref_bytes}, {num_live, 4}, {device_status, 4},
                              {workspace, mqa::compact_workspace_bytes(num_blocks)}};
    const ApiSpan reads[] = {{block_table == new_table ? nullptr : block_table, table}, {seq_lens, rows * 4ull},
                             {refs == new_refs ? nullptr : refs, ref_bytes}};
    if (mqa::api_clash(writes, reads) || places.hold_any(writes) || places.hold_any(reads)) return MQA_ERR_INVALID_ARG;
    if (!api_aligned(workspace, 16)) return MQA_ERR_INVALID_ARG;
    const int sms = mqa::api_sm_count();
    if (sms < 1) return MQA_ERR_CUDA;
    mqa::PagesArgs a{};
    a.table = block_table;
    a.lens = seq_lens;
    a.refs = refs;
    a.new_table = new_table;
    a.new_refs = new_refs;
    a.moved = moved;
    a.num_live = num_live;
    a.ws = static_cast<int32_t*>(workspace);
    a.status = device_status;
    a.rows = a.new_rows = rows;
    a.width = max_blocks;
    a.num_blocks = num_blocks;
    a.page = page_size;
    const cudaError_t e = mqa::pages_compact(a, pools, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MQA_OK : api_cuda_fail(e);
}

}  // extern "C"

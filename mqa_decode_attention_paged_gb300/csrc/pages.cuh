// Forking and compacting the pages of paged caches: arguments and the host
// interface.
#pragma once

#include "common.cuh"

namespace mqa {

constexpr int kMaxPools = 256;
constexpr int kPagesMaxRows = 8192;

// The tensors whose first dimension is a page, one after the other in chunks.
// They go to the kernel by value; kFewPools of them in a structure of their own,
// as a launch with the 5 KB of the large one takes 4 us longer on the host.
constexpr int kFewPools = 16;
template <int N>
struct PoolsOf {
    struct Pool {
        char* base;
        long long bytes;  // of a page, a multiple of 4
    } pool[N];
    int first[N + 1];  // chunks of a page before each
    int n;
};
using PagePools = PoolsOf<kMaxPools>;

struct PagesArgs {
    const int32_t* table;    // [rows, width]
    const int32_t* lens;     // [rows]
    const int32_t* parents;  // [new_rows] (fork)
    const int32_t* refs;     // [num_blocks]
    int32_t* new_table;      // [new_rows, width]
    int32_t* new_lens;       // [new_rows] (fork)
    int32_t* new_refs;       // [num_blocks]
    int32_t* moved;          // [num_blocks] (compact)
    int32_t* num_live;       // (compact)
    int32_t* ws;             // header, then lists (see pages.cu)
    int* status;
    int rows, new_rows, width, num_blocks, page;
};

constexpr int kPageChunk = 32 * 1024;  // bytes that a thread block copies at a time
constexpr int kPagesHeader = 64;       // ints before the lists

inline size_t fork_workspace_bytes(int new_rows) { return (kPagesHeader + 3ull * new_rows) * 4; }
inline size_t compact_workspace_bytes(int num_blocks) { return (kPagesHeader + 3ull * num_blocks) * 4; }

cudaError_t pages_fork(const PagesArgs& a, const PagePools& pools, int sms, cudaStream_t stream);
cudaError_t pages_compact(const PagesArgs& a, const PagePools& pools, int sms, cudaStream_t stream);

}  // namespace mqa

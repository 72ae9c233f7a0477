// Forking and compacting the pages of paged caches.
//
// Fork: new row r is a copy of row parents[r] (none if it is -1).  With c(p) the
// children of row p, a full page of p gains c(p) - 1 holders; a partly filled
// last page stays with the first child, so it gains (c(p) > 0) - 1, and every
// other child gets a page of its own, the lowest free ones in the order of the
// rows, with a copy of its data.  Pages whose count falls to 0 are free, for this
// call's children too (what is copied from has a holder, so nothing is
// overwritten).
// Compact: with L live pages (count > 0), the live pages with ids >= L move, in
// ascending order, to the free ids < L.
//
// Both are bound by the copies (2 bytes of traffic a byte of page; HBM), and
// where there are few by the chain of dependent steps.  So a call is two
// launches: a plan by one cluster of eight thread blocks, which meet at the
// cluster's barrier between the steps, and a copy by the whole device, which
// writes the table as well.  Counts are changed by integer atomics and free
// pages numbered by prefix sums: the result does not depend on any order.
//
// Measured: 64 prompts forked 8 ways over 6 layers of e4m3 caches (352 MB written) 85
// us, of them 12 the plan; compacting 256 rows over two layers of bf16 caches (318 MB
// moved) 112 us, 84 % of a copy's rate.  8 beams of 4 over one layer 10 us on the GPU and 25
// to 30 from Python, which is the host's part (allocation 10, the C call 5).
#include "pages.cuh"

#include <atomic>

namespace mqa {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
// header of the workspace
constexpr int kPairs = 0, kCounts = 16, kCounts2 = 32;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Meets the cluster's other blocks; what they wrote to global memory before is visible after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Loads that see what other blocks of the cluster wrote (not the read-only path).
__device__ __forceinline__ int ld(const int32_t* p) {
    int v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Exclusive prefix sum over the block's threads; the total in `all`.
__device__ __forceinline__ int block_scan(int* scratch, int v, int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp ? before : 0) + x - v;
}

// Length of a row, within its table.
__device__ __forceinline__ int row_len(const PagesArgs& a, int p, int* status) {
    const int n = __ldg(a.lens + p);
    const long long cap = static_cast<long long>(a.width) * a.page;
    if (n < 0 || n > cap) {
        report(status, MQA_ERR_DEVICE_CHECK);
        return n < 0 ? 0 : static_cast<int>(cap);
    }
    return n;
}
__device__ __forceinline__ int pages_of(const PagesArgs& a, int n) { return n / a.page + (n % a.page != 0); }
__device__ __forceinline__ bool is_page(const PagesArgs& a, int id) { return id >= 0 && id < a.num_blocks; }
__device__ __forceinline__ int parent_of(const PagesArgs& a, int r, int* status) {
    const int p = __ldg(a.parents + r);
    if (p < -1 || p >= a.rows) {
        report(status, MQA_ERR_DEVICE_CHECK);
        return -1;
    }
    return p;
}

// The part of [0, num_blocks) that block `rank` of the cluster looks after: ids from lo on, four a thread a turn.
__device__ __forceinline__ void share(const PagesArgs& a, int rank, int& lo, int& hi) {
    const int per = (a.num_blocks + kCluster - 1) / kCluster;
    lo = min(a.num_blocks, rank * per);
    hi = min(a.num_blocks, lo + per);
}
constexpr int kIds = 4;

// Workspace after the header: pairs' sources [new_rows], destinations [new_rows], own page of each new row
// (-1: could not be had, -2: shares its parent's) [new_rows].
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const __grid_constant__ PagesArgs a) {
    extern __shared__ int smem[];
    int* children = smem;           // [rows]
    int* first = smem + a.rows;     // [rows]
    __shared__ int scratch[32];
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_rank());
    int32_t* src = a.ws + kPagesHeader;
    int32_t* dst = src + a.new_rows;
    int32_t* own = dst + a.new_rows;
    int lo, hi;
    share(a, rank, lo, hi);
    for (int p = tid; p < a.rows; p += kThreads) {
        children[p] = 0;
        first[p] = a.new_rows;
    }
    pdl_wait();
    pdl_launch_dependents();
    for (int i = lo + tid; i < hi; i += kThreads) a.new_refs[i] = __ldg(a.refs + i);
    __syncthreads();
    for (int r = tid; r < a.new_rows; r += kThreads) {
        const int p = parent_of(a, r, rank == 0 ? a.status : nullptr);
        if (p < 0) continue;
        atomicAdd(&children[p], 1);
        atomicMin(&first[p], r);
    }
    __syncthreads();
    cluster_sync();  // the counts are copied

    // changes of the counts: a warp a row
    for (int p = rank * (kThreads / 32) + (tid >> 5); p < a.rows; p += kCluster * (kThreads / 32)) {
        const int n = row_len(a, p, a.status), c = children[p];
        if (c == 1) continue;
        const int k = pages_of(a, n), tail = n % a.page ? k - 1 : -1;
        for (int j = tid & 31; j < k; j += 32) {
            const int id = __ldg(a.table + static_cast<long long>(p) * a.width + j);
            if (!is_page(a, id))
                report(a.status, MQA_ERR_DEVICE_CHECK);
            else if (const int change = j == tail ? (c > 0) - 1 : c - 1; change != 0)
                atomicAdd(a.new_refs + id, change);
        }
    }
    // which rows need a page of their own, numbered (by the last block, which has the fewest ids at most)
    if (rank == kCluster - 1) {
        int base = 0;
        for (int r0 = 0; r0 < a.new_rows; r0 += kThreads) {
            const int r = r0 + tid;
            int need = 0, last = -1;
            if (r < a.new_rows) {
                const int p = parent_of(a, r, nullptr), n = p < 0 ? 0 : row_len(a, p, nullptr);
                a.new_lens[r] = n;
                if (p >= 0 && n % a.page != 0 && first[p] != r) {
                    last = __ldg(a.table + static_cast<long long>(p) * a.width + n / a.page);
                    need = is_page(a, last);
                }
            }
            int all;
            const int at = base + block_scan(scratch, need, all);
            if (need) src[at] = last;
            if (r < a.new_rows) own[r] = need ? at : -2;  // (the number for now)
            base += all;
        }
        if (tid == 0) a.ws[kPairs] = base;
    }
    cluster_sync();  // counts are final, the needs known

    const int needs = ld(a.ws + kPairs);
    int free_here = 0;
    if (needs > 0)
        for (int i = lo + tid; i < hi; i += kThreads) free_here += ld(a.new_refs + i) == 0;
    int all;
    block_scan(scratch, free_here, all);
    if (tid == 0) a.ws[kCounts + rank] = all;
    cluster_sync();
    int at = 0, total = 0;
    for (int k = 0; k < kCluster; ++k) {
        const int c = ld(a.ws + kCounts + k);
        if (k < rank) at += c;
        total += c;
    }
    for (int i0 = lo; i0 < hi && at < needs; i0 += kThreads * kIds) {
        const int i = i0 + tid * kIds;
        int v[kIds], mine = 0;
#pragma unroll
        for (int e = 0; e < kIds; ++e) {
            v[e] = i + e < hi ? ld(a.new_refs + i + e) : 1;
            mine += v[e] == 0;
        }
        int k = at + block_scan(scratch, mine, all);
#pragma unroll
        for (int e = 0; e < kIds; ++e)
            if (v[e] == 0) {
                if (k < needs) {
                    dst[k] = i + e;
                    a.new_refs[i + e] = 1;
                }
                ++k;
            }
        at += all;
    }
    cluster_sync();
    if (rank == 0) {
        if (needs > total && tid == 0) {
            report(a.status, MQA_ERR_DEVICE_CHECK);
            a.ws[kPairs] = total;
        }
        for (int r = tid; r < a.new_rows; r += kThreads) {
            const int k = ld(own + r);
            if (k >= 0) own[r] = k < total ? ld(dst + k) : -1;
        }
    }
}

// Workspace after the header: sources [num_blocks], destinations [num_blocks], counts of the sources [num_blocks].
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ int scratch[32];
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_rank());
    int32_t* src = a.ws + kPagesHeader;
    int32_t* dst = src + a.num_blocks;
    int32_t* src_refs = dst + a.num_blocks;
    int lo, hi;
    share(a, rank, lo, hi);
    pdl_wait();
    pdl_launch_dependents();
    int n = 0, all;
    for (int i = lo + tid; i < hi; i += kThreads) n += ld(a.refs + i) > 0;
    block_scan(scratch, n, all);
    if (tid == 0) a.ws[kCounts + rank] = all;
    cluster_sync();
    int before = 0, live = 0;  // live pages of the shares before, of all
    for (int k = 0; k < kCluster; ++k) {
        const int c = ld(a.ws + kCounts + k);
        if (k < rank) before += c;
        live += c;
    }
    n = 0;
    for (int i = lo + tid; i < min(hi, live); i += kThreads) n += ld(a.refs + i) > 0;
    block_scan(scratch, n, all);
    if (tid == 0) a.ws[kCounts2 + rank] = all;
    cluster_sync();
    int stay = 0;  // live pages with an id below `live`
    for (int k = 0; k < kCluster; ++k) stay += ld(a.ws + kCounts2 + k);
    // twice over the share: the lists, then what follows from them
    for (int turn = 0; turn < 2; ++turn) {
        int at = before;
        for (int i0 = lo; i0 < hi; i0 += kThreads * kIds) {
            const int i = i0 + tid * kIds;
            int v[kIds], mine = 0;
#pragma unroll
            for (int e = 0; e < kIds; ++e) {
                v[e] = i + e < hi ? ld(a.refs + i + e) : 0;
                mine += v[e] > 0;
            }
            int k = at + block_scan(scratch, mine, all);  // live pages before i + e
#pragma unroll
            for (int e = 0; e < kIds; ++e) {
                const int id = i + e;
                if (id >= hi) break;
                const bool lives = v[e] > 0;
                if (turn == 0) {
                    if (!lives && id < live) dst[id - k] = id;
                    if (lives && id >= live) {
                        src[k - stay] = id;
                        src_refs[k - stay] = v[e];
                    }
                } else {
                    a.moved[id] = !lives ? -1 : id < live ? id : ld(dst + k - stay);
                    a.new_refs[id] = id < live ? (lives ? v[e] : ld(src_refs + id - k)) : (lives ? 0 : v[e]);
                }
                k += lives;
            }
            at += all;
        }
        if (turn == 0) cluster_sync();
    }
    if (rank == 0 && tid == 0) {
        a.ws[kPairs] = live - stay;
        *a.num_live = live;
    }
}

// ---- copies
constexpr int kCopyThreads = 256;
constexpr int kCopyCtasPerSm = 4;

// The pairs' pages in every pool, chunk by chunk.
template <int N>
__device__ __forceinline__ void copy_pairs(const PoolsOf<N>& pools, const int32_t* src, const int32_t* dst, int pairs) {
    const int per = pools.first[pools.n];
    const long long items = static_cast<long long>(pairs) * per;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int pair = static_cast<int>(item / per), c = static_cast<int>(item - static_cast<long long>(pair) * per);
        int lo = 0, hi = pools.n - 1;  // the pool that chunk c lies in
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pools.first[mid] <= c)
                lo = mid;
            else
                hi = mid - 1;
        }
        const long long bytes = pools.pool[lo].bytes, off = static_cast<long long>(c - pools.first[lo]) * kPageChunk;
        const int len = static_cast<int>(min(static_cast<long long>(kPageChunk), bytes - off));
        const char* s = pools.pool[lo].base + src[pair] * bytes + off;
        char* d = pools.pool[lo].base + dst[pair] * bytes + off;
        if (bytes % 16 == 0) {
            constexpr int kInFlight = kPageChunk / 16 / kCopyThreads;
            uint4 v[kInFlight];
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int i = (k * kCopyThreads + threadIdx.x) * 16;
                if (i < len) v[k] = __ldcs(reinterpret_cast<const uint4*>(s + i));
            }
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int i = (k * kCopyThreads + threadIdx.x) * 16;
                if (i < len) __stcs(reinterpret_cast<uint4*>(d + i), v[k]);
            }
        } else {  // (pages that do not start on 16 bytes: small ones, as of block scales)
            for (int i = threadIdx.x * 4; i < len; i += kCopyThreads * 4)
                *reinterpret_cast<uint32_t*>(d + i) = *reinterpret_cast<const uint32_t*>(s + i);
        }
    }
}

template <bool FORK, int N>
__global__ void __launch_bounds__(kCopyThreads, kCopyCtasPerSm)
    pages_copy_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PoolsOf<N> pools) {
    pdl_wait();
    pdl_launch_dependents();
    const int32_t* src = a.ws + kPagesHeader;
    const int32_t* dst = src + (FORK ? a.new_rows : a.num_blocks);
    // the table: a block a row at a time, the last ones first (the first have the most to copy)
    for (int r = static_cast<int>(gridDim.x) - 1 - blockIdx.x; r < a.new_rows; r += gridDim.x) {
        int32_t* out = a.new_table + static_cast<long long>(r) * a.width;
        if constexpr (FORK) {
            const int p = parent_of(a, r, nullptr);
            const int n = p < 0 ? 0 : row_len(a, p, nullptr), k = pages_of(a, n);
            const int own = dst[a.new_rows + r];  // own pages lie after the destinations
            const int32_t* in = a.table + static_cast<long long>(p < 0 ? 0 : p) * a.width;
            for (int j = threadIdx.x; j < a.width; j += kCopyThreads) {
                int id = -1;
                if (j < k) {
                    id = __ldg(in + j);
                    if (!is_page(a, id)) report(a.status, MQA_ERR_DEVICE_CHECK);  // (kept; the plan does not look at rows with one child)
                    if (j == k - 1 && own != -2) id = own;
                }
                out[j] = id;
            }
        } else {
            const int k = pages_of(a, row_len(a, r, a.status));
            const int32_t* in = a.table + static_cast<long long>(r) * a.width;
            for (int j = threadIdx.x; j < a.width; j += kCopyThreads) {
                const int id = in[j];
                int to = id;
                if (j < k) {
                    to = is_page(a, id) ? a.moved[id] : -1;
                    if (to < 0) {  // not a live page: as it is
                        report(a.status, MQA_ERR_DEVICE_CHECK);
                        to = id;
                    }
                }
                out[j] = to;
            }
        }
    }
    if (pools.n > 0) copy_pairs(pools, src, dst, a.ws[kPairs]);
}

cudaError_t launch_plan(void (*kern)(PagesArgs), const PagesArgs& a, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool FORK>
cudaError_t launch_copy(const PagesArgs& a, const PagePools& pools, int sms, cudaStream_t stream) {
    const dim3 grid(sms * kCopyCtasPerSm), block(kCopyThreads);
    if (pools.n > kFewPools) return launch_with_pdl(pages_copy_kernel<FORK, kMaxPools>, grid, block, 0, stream, a, pools);
    PoolsOf<kFewPools> few;
    for (int i = 0; i < pools.n; ++i) few.pool[i] = {pools.pool[i].base, pools.pool[i].bytes};
    for (int i = 0; i <= pools.n; ++i) few.first[i] = pools.first[i];
    few.n = pools.n;
    return launch_with_pdl(pages_copy_kernel<FORK, kFewPools>, grid, block, 0, stream, a, few);
}

}  // namespace

cudaError_t pages_fork(const PagesArgs& a, const PagePools& pools, int sms, cudaStream_t stream) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (!known || !done[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * kPagesMaxRows * static_cast<int>(sizeof(int)));
        if (e != cudaSuccess) return e;
        if (known) done[dev].store(true, std::memory_order_relaxed);
    }
    if (cudaError_t e = launch_plan(fork_plan_kernel, a, 2 * sizeof(int) * a.rows, stream); e != cudaSuccess) return e;
    return launch_copy<true>(a, pools, sms, stream);
}

cudaError_t pages_compact(const PagesArgs& a, const PagePools& pools, int sms, cudaStream_t stream) {
    if (cudaError_t e = launch_plan(compact_plan_kernel, a, 0, stream); e != cudaSuccess) return e;
    return launch_copy<false>(a, pools, sms, stream);
}

}  // namespace mqa

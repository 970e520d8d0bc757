// Shared by the paged-cache kernels (append, attend, evict): the cache's device view.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvp.h"
#include "kvp_internal.cuh"

namespace kvp {

constexpr int kMaxCacheRows = 1 << 23;    // M * P (the eviction counts a warp's rows in 16 bits)
constexpr int kMaxCacheHeads = 1 << 20;   // b * hkv
constexpr int kMaxCacheGroup = 64;        // G

// Whether the shape is inside kvp.h's limits.
inline bool cache_shape_ok(const kvp_cache_shape& s) {
    if (s.batch < 1 || s.hkv < 1 || s.hq < 1 || s.hq % s.hkv != 0) return false;
    if ((long long)s.batch * s.hkv > kMaxCacheHeads || s.hq / s.hkv > kMaxCacheGroup) return false;
    if (s.head_dim != 64 && s.head_dim != 128) return false;
    if (s.page_size < 16 || s.page_size > 256 || (s.page_size & (s.page_size - 1)) != 0) return false;
    if (s.num_pages < 1 || s.max_pages < 1 || (long long)s.max_pages * s.page_size > kMaxCacheRows) return false;
    return s.dtype == KVP_BF16 || s.dtype == KVP_FP16;
}

inline int log2_of(int pow2) {
    int n = 0;
    while ((1 << n) < pow2) ++n;
    return n;
}

// The page table and lengths of a cache on the device. A head is a (sequence, KV head).
struct CacheView {
    const int32_t* table;    // [heads][max_pages]
    const int32_t* lens;     // [heads]
    int heads, max_pages, num_pages, page_shift;

    __host__ __device__ __forceinline__ int cap() const { return max_pages << page_shift; }
    // Plain loads, not the read-only path: the stream's previous kernel may have written them
    // while this one was already resident (programmatic dependent launch).
    __device__ __forceinline__ int len(int head) const { return min(max(lens[head], 0), cap()); }
    // The pool's row that holds row j of `head` (0 <= j < cap), or -1 if it has no page.
    __device__ __forceinline__ long long row(int head, int j) const {
        const int page = table[(size_t)head * max_pages + (j >> page_shift)];
        if (page < 0 || page >= num_pages) return -1;
        return ((long long)page << page_shift) + (j & ((1 << page_shift) - 1));
    }
};

inline CacheView cache_view(const kvp_cache_shape& s, const int32_t* table, const int32_t* lens) {
    CacheView c;
    c.table = table;
    c.lens = lens;
    c.heads = s.batch * s.hkv;
    c.max_pages = s.max_pages;
    c.num_pages = s.num_pages;
    c.page_shift = log2_of(s.page_size);
    return c;
}

// Launches (each returns the launch's cudaError_t), and their workspaces.
size_t attend_workspace_bytes(const kvp_cache_shape& s, bool accumulate);   // 0: too many tiles
cudaError_t launch_attend(const kvp_cache_shape& s, const uint16_t* q, const uint16_t* k_pages,
                          const uint16_t* v_pages, const int32_t* table, const int32_t* lens, uint16_t* out,
                          float* lse, float* acc, void* workspace, cudaStream_t st);
cudaError_t launch_append(const kvp_cache_shape& s, const uint16_t* k_new, const uint16_t* v_new, int n,
                          const int32_t* counts, const float* weight, uint16_t* k_pages, uint16_t* v_pages,
                          float* acc, const int32_t* table, const int32_t* lens, int32_t* lens_out,
                          cudaStream_t st);
size_t evict_workspace_bytes(const kvp_cache_shape& s, const kvp_evict& e);
cudaError_t launch_evict(const kvp_cache_shape& s, const kvp_evict& e, const int32_t* budgets,
                         uint16_t* k_pages, uint16_t* v_pages, const float* acc, float* acc_out,
                         const int32_t* table, const int32_t* lens, int32_t* lens_out, int32_t* src,
                         void* workspace, cudaStream_t st);

// A launch on `st` that may start while the stream's previous kernel runs out (programmatic
// dependent launch): the kernel calls ptx::grid_dependency_wait() before it touches memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), int grid, int block, size_t smem, cudaStream_t st,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

}  // namespace kvp

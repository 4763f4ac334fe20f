// selected.cuh -- serving with selected pages: parameters and launchers of the
// tables, token-append, page-bounds, selection and selected-attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"

namespace pkv {

// The dynamic shared memory that a kernel may ask for, set once a device.
struct SmemLimit {
    std::atomic<uint64_t> done{0};  // bit per device
    cudaError_t set(const void* fn, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// SMs of the current device (at least 1).
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return 1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

constexpr int kMaxTableBatch = 16384;    // requests of one paged_tables_build
constexpr int kMaxAppendRows = 4096;     // rows of a token (q, k, v) of one kv_append_tokens
constexpr int kMaxSelectPages = 131072;  // table columns of one paged_select_pages
constexpr int kSelectTile = 64;          // the fewest pages of a score CTA of paged_select_pages
constexpr int kMaxSelectGroup = 192;     // query heads of a KV head: their rows in shared memory

// Thread-block clusters.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct TablesArgs {
    const int32_t* cached;      // [B]
    const int32_t* fresh;       // [B] new tokens
    int batch;
    const int32_t* free_pages;  // [n_free]
    int n_free;
    const int32_t* free_begin;  // nullable: 0
    int32_t* free_end;
    int page_size, num_pages;
    int32_t* table;
    int table_stride;
    int32_t* lens;              // [B]
    int32_t* starts;            // [B + 1]
    int n_tokens;
    int32_t* positions;         // [n_tokens]
    int32_t* seq_ids;
    int64_t* slots;
    uint32_t* status;
};
cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream);

struct AppendTokensArgs {
    const void* q;  // null: no queries
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
    const int64_t* slots;
    const int32_t* positions;  // null: no rotation
    int n_tokens, n_q_heads, n_kv_heads, page_size;
    long long n_slots;         // num_pages * page_size
    void* k_pool;
    void* v_pool;
    void* q_out;
    const void* q_norm;
    const void* k_norm;
    float eps;
    uint32_t* status;
    pkv_rope rope;
};
cudaError_t launch_append_tokens(const AppendTokensArgs& a, bool bf16, int head_dim,
                                 cudaStream_t stream);

struct BoundsArgs {
    const void* k_pool;
    const int64_t* slots;
    int n_tokens, n_kv_heads, page_size;
    long long n_slots;
    void* bounds;
    uint32_t* status;
};
cudaError_t launch_page_bounds(const BoundsArgs& a, bool bf16, int head_dim, cudaStream_t stream);

struct SelectArgs {
    const void* q;
    const void* bounds;  // [NP][Hkv][2][D]
    const int32_t* table;
    int table_stride;
    const int32_t* lens;
    int batch, n_q_heads, n_kv_heads, page_size, num_pages;
    int keep_first, keep_last, max_pages;
    int32_t* selected;   // [B][Hkv][max_pages]
    unsigned long long* keys64;  // workspace [B][Hkv][stride]: 64-bit scores, as ordered keys
    float* scores;       // workspace [B][Hkv][stride]
    uint4* stats;        // workspace [B][Hkv][tiles]: what a tile of scores leaves for the choice
    int tiles, tile_pages;  // a score CTA takes tile_pages pages (set by the launch)
    uint32_t* status;
};
cudaError_t launch_select(const SelectArgs& a, bool bf16, int head_dim, cudaStream_t stream);

struct SelectedParams {
    const void* q;
    const int32_t* table;
    int table_stride;
    const int32_t* lens;
    const int32_t* selected;  // [B][Hkv][max_pages]
    int max_pages;
    int batch, n_q_heads, n_kv_heads, page_size, num_pages;
    int group, head_blocks;   // head blocks of at most 16 query heads
    float scale_log2;
    void* out;
    uint32_t* status;
};
cudaError_t launch_selected(const SelectedParams& p, bool bf16, int head_dim,
                            const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream);

// The tensor map of a pool's rows (16-row boxes, api.cu).
pkv_status pool_rows_map(const void* pool, long long rows, int head_dim, pkv_dtype dtype,
                         CUtensorMap* out);

}  // namespace pkv

// kda_linear.h -- host-side interface of the linear-attention and cache-page kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct LinearStepParams {
    int N, H, group;                  // group = value heads per query / key head
    const void *q, *k, *v;            // [N, H / group, Dk], [N, H / group, Dk], [N, H, Dv]
    const float *g;                   // [N, H], or [H] when g_per_head
    int g_per_head;
    float scale;
    const int32_t *slots;             // [N] or null
    int n_slots;
    const float *state;               // [n_slots, H, Dk, Dv]
    float *new_state;                 // may equal state
    void *o;                          // [N, H, Dv]
};

hipError_t launch_linear_step(int bf16, int Dk, int Dv, const LinearStepParams &p, hipStream_t stream);

// One pool of pages; unit: widest access (16, 4, 2 or 1 bytes) that its base
// addresses and page size allow.
struct CachePool {
    char *dst;
    const char *src;
    size_t page_bytes;
    int unit;
    int slices;                       // workgroup-sized pieces of a page
};

constexpr int CACHE_MAX_POOLS = 8;
constexpr size_t CACHE_SLICE = 32768; // bytes one workgroup copies

struct CachePools {
    CachePool pool[CACHE_MAX_POOLS];
    int n;
    int slices;                       // over all pools
};

hipError_t launch_cache_copy(const CachePools &pools, int n_dst, int n_src, const int32_t *dst_pages,
                             const int32_t *src_pages, int n, hipStream_t stream);
hipError_t launch_cache_fork(const CachePools &pools, int n_pages, int32_t *table, int rows, int per_row,
                             int32_t *refcount, const int32_t *parents, const int32_t *children, int n,
                             int32_t *old_pages, int32_t *new_pages, hipStream_t stream);
hipError_t launch_cache_free(int32_t *table, int rows, int per_row, int32_t *refcount, int n_pages,
                             const int32_t *free_rows, int n, hipStream_t stream);
hipError_t launch_cache_compact(const CachePools &pools, int n_pages, int32_t *table, int rows, int per_row,
                                int32_t *refcount, int32_t *moved_to, int32_t *moves, int32_t *counts,
                                hipStream_t stream);

}  // namespace kda

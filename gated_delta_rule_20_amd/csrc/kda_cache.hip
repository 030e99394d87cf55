// kda_cache.hip -- pages of a state cache: copying, forking, freeing, compacting.
//
// Page contents are moved once, from their place to their new one, in 16-byte
// accesses where base and page size allow; that is bound by HBM (two passes over
// the page bytes).  The tables are a few KiB: planning is one workgroup's work
// and costs a launch, not bandwidth (5 us for 512 pages, 6 us for 8 forks).  Copies run at 5.3 TB/s
// (256 pages of 2.1 MiB), compaction's moves at 5.2 TB/s.  Every result depends on the arguments
// alone: ties go to the lowest index, counts are integer sums.
#include "kda_common.h"
#include "kda_linear.h"

namespace kda {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// bytes [begin, end) of one page in accesses of U, by 256 threads, eight of each
// in flight; go() is asked once, by every thread, between the first loads and the
// first stores.
template <typename U, typename F>
__device__ __forceinline__ void copy_range(char *dst, const char *src, size_t begin, size_t end, F go)
{
    const U *s = reinterpret_cast<const U *>(src + begin);
    U *d = reinterpret_cast<U *>(dst + begin);
    const unsigned n = (unsigned)((end - begin) / sizeof(U)), t = threadIdx.x;
    U x[8];
    const auto load = [&](unsigned base) {
#pragma unroll
        for (unsigned j = 0; j < 8; ++j)
            if (base + t + j * 256 < n) x[j] = __builtin_nontemporal_load(s + base + t + j * 256);
    };
    load(0);
    if (!go()) return;
    for (unsigned base = 0;;) {
#pragma unroll
        for (unsigned j = 0; j < 8; ++j)
            if (base + t + j * 256 < n) __builtin_nontemporal_store(x[j], d + base + t + j * 256);
        base += 8 * 256;
        if (base >= n) break;
        load(base);
    }
}

// One slice (of pools.slices) of page `from` to page `to`.
template <typename F> __device__ __forceinline__ void copy_slice(const CachePools &pools, int slice, int from, int to, F go)
{
    // Which pool the slice is of.  Field by field, without a variable index: that would put the kernel's arguments into
    // scratch memory, at every workgroup's start (without it 2000 pages of 17 KiB take 15 us).
    char *dst = pools.pool[0].dst;
    const char *src = pools.pool[0].src;
    size_t bytes = pools.pool[0].page_bytes;
    int unit = pools.pool[0].unit, slices = pools.pool[0].slices;
#pragma unroll
    for (int i = 1; i < CACHE_MAX_POOLS; ++i) {
        const bool next = slice >= slices;
        slice -= next ? slices : 0;
        dst = next ? pools.pool[i].dst : dst;
        src = next ? pools.pool[i].src : src;
        bytes = next ? pools.pool[i].page_bytes : bytes;
        unit = next ? pools.pool[i].unit : unit;
        slices = next ? pools.pool[i].slices : slices;
    }
    const size_t begin = (size_t)slice * CACHE_SLICE;
    const size_t end = min(begin + CACHE_SLICE, bytes);
    dst += (size_t)to * bytes;
    src += (size_t)from * bytes;
    switch (unit) {
    case 16: copy_range<u32x4>(dst, src, begin, end, go); break;
    case 4: copy_range<uint32_t>(dst, src, begin, end, go); break;
    case 2: copy_range<uint16_t>(dst, src, begin, end, go); break;
    default: copy_range<uint8_t>(dst, src, begin, end, go); break;
    }
}
__device__ __forceinline__ bool always() { return true; }

// One workgroup per (pair, slice).
__global__ __launch_bounds__(256) void cache_copy_kernel(const CachePools pools, int n_dst, int n_src,
                                                         const int32_t *__restrict__ dst_pages,
                                                         const int32_t *__restrict__ src_pages, int n)
{
    const int i = (int)(blockIdx.x / (unsigned)pools.slices), slice = (int)(blockIdx.x % (unsigned)pools.slices);
    const int to = dst_pages[i], from = src_pages[i];
    if (to < 0 || to >= n_dst || from < 0 || from >= n_src) return;
    copy_slice(pools, slice, from, to, [&]() {
        bool again = false;                   // a later pair has this destination
        for (long j = i + 1 + (long)threadIdx.x; j < n; j += 8 * 256) {   // eight reads in flight
            int d[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) d[m] = dst_pages[min(j + 256 * m, (long)n - 1)];
#pragma unroll
            for (int m = 0; m < 8; ++m)
                if (d[m] == to && j + 256 * m < n) {
                    const int s = src_pages[j + 256 * m];
                    again |= s >= 0 && s < n_src;
                }
        }
        return !__syncthreads_or(again);
    });
}

// The copies a fork planned: old_pages[i] to new_pages[i] (-1: none).
__global__ __launch_bounds__(256) void cache_fork_copy_kernel(const CachePools pools,
                                                              const int32_t *__restrict__ old_pages,
                                                              const int32_t *__restrict__ new_pages)
{
    const int i = (int)(blockIdx.x / (unsigned)pools.slices), slice = (int)(blockIdx.x % (unsigned)pools.slices);
    const int from = old_pages[i], to = new_pages[i];
    if (from < 0 || to < 0) return;
    copy_slice(pools, slice, from, to, always);
}

constexpr int PLAN = 1024;                    // threads of a planning workgroup

// Exclusive prefix sum of v over the workgroup; total in every thread.  s: one
// int per wave.  Ends with a barrier, so it may be called in a loop.
__device__ __forceinline__ int block_prefix(int v, int *s, int &total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 63) s[w] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < PLAN / 64; ++i) {
        before += i < w ? s[i] : 0;
        total += s[i];
    }
    __syncthreads();
    return before + x - v;
}

constexpr int FORK_INVALID = -2, FORK_EMPTY = -1;

// Plans and books a fork call.  old_pages / new_pages hold the plan while it is
// made: first old_pages[i] = does fork i need a page, then its rank among those
// that do; new_pages = the free pages by rank, then each fork's page.
__global__ __launch_bounds__(PLAN) void cache_fork_plan_kernel(int n_pages, int32_t *table, int rows, int per_row,
                                                               int32_t *refcount, const int32_t *__restrict__ parents,
                                                               const int32_t *__restrict__ children, int n,
                                                               int32_t *old_pages, int32_t *new_pages)
{
    __shared__ int s_sum[PLAN / 64];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    // 1. one wave per fork: is it allowed, and does its parent hold a page
    for (int i = w; i < n; i += PLAN / 64) {
        const int a = parents[i], c = children[i];
        bool bad = a < 0 || a >= rows || c < 0 || c >= rows;
        for (int j = lane; j < n; j += 64) bad |= parents[j] == c || (j < i && children[j] == c);
        bad = __any(bad);
        bool any = false;
        if (!bad)
            for (int j = lane; j < per_row; j += 64) {
                const int p = table[(size_t)a * per_row + j];
                any |= p >= 0 && p < n_pages;
            }
        any = __any(any);
        if (lane == 0) old_pages[i] = bad ? FORK_INVALID : any ? 1 : FORK_EMPTY;
    }
    __syncthreads();
    // 2. ranks
    int wanted = 0;
    for (int b = 0; b < n; b += PLAN) {
        const int i = b + t;
        const int need = i < n && old_pages[i] == 1;
        int total;
        const int r = block_prefix(need, s_sum, total);
        if (need) old_pages[i] = wanted + r;
        wanted += total;
    }
    // 3. the lowest free pages, by rank (at most n of them)
    int found = 0;
    for (int b = 0; b < n_pages && found < wanted; b += 4 * PLAN) {
        int p = b + 4 * t, f[4], sum = 0, total;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = p + j < n_pages && refcount[p + j] <= 0;
            sum += f[j];
        }
        int r = found + block_prefix(sum, s_sum, total);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (f[j] && r < wanted) new_pages[r] = p + j;
            r += f[j];
        }
        found += total;
    }
    found = min(found, wanted);
    __syncthreads();
    // 4. each fork's page, from the last fork down: rank <= fork, so no entry is overwritten before it is read
    for (int b = (n - 1) / PLAN * PLAN; b >= 0; b -= PLAN) {
        const int i = b + t;
        int page = -1;
        if (i < n && old_pages[i] >= 0 && old_pages[i] < found) page = new_pages[old_pages[i]];
        __syncthreads();
        if (i < n) new_pages[i] = page;
        __syncthreads();
    }
    // 5. one wave per fork: the child's row and the counts
    for (int i = w; i < n; i += PLAN / 64) {
        const int state = old_pages[i], page = new_pages[i];
        int last = -1;
        if (state != FORK_INVALID) {
            const int32_t *from = table + (size_t)parents[i] * per_row;
            int32_t *to = table + (size_t)children[i] * per_row;
            for (int j = lane; j < per_row; j += 64) last = (from[j] >= 0 && from[j] < n_pages) ? j : last;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) last = max(last, __shfl_xor(last, d));
            for (int j = lane; j < per_row; j += 64) {
                const int p = from[j];
                const bool held = page >= 0 && p >= 0 && p < n_pages && j < last;
                if (held) atomicAdd(&refcount[p], 1);
                to[j] = held ? p : (page >= 0 && j == last) ? page : -1;
            }
            if (page >= 0 && lane == 0) atomicExch(&refcount[page], 1);
            last = page >= 0 ? from[last] : -1;
        }
        if (lane == 0) old_pages[i] = last;
    }
}

// One thread per table entry of the freed rows.
__global__ __launch_bounds__(256) void cache_free_kernel(int32_t *table, int rows, int per_row, int32_t *refcount,
                                                         int n_pages, const int32_t *__restrict__ free_rows, int n)
{
    const size_t total = (size_t)n * per_row;
    for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (size_t)gridDim.x * 256) {
        const int r = free_rows[e / per_row];
        if (r < 0 || r >= rows) continue;
        // whoever takes the entry gives up its page, so a row named twice is freed once
        const int p = atomicExch(&table[(size_t)r * per_row + e % per_row], -1);
        if (p < 0 || p >= n_pages) continue;
        if (atomicSub(&refcount[p], 1) <= 0) atomicAdd(&refcount[p], 1);   // not below 0
    }
}

// counts[0] = live pages, counts[1] = moves; moves[2 r], moves[2 r + 1] = from, to.
__global__ __launch_bounds__(PLAN) void cache_compact_plan_kernel(int n_pages, int32_t *refcount, int32_t *moved_to,
                                                                  int32_t *moves, int32_t *counts)
{
    __shared__ int s_sum[PLAN / 64];
    const int t = threadIdx.x;
    int mine = 0, n_live;
    for (int p = t; p < n_pages; p += PLAN) mine += refcount[p] > 0;
    block_prefix(mine, s_sum, n_live);
    int holes = 0, movers = 0;
    for (int b = 0; b < n_pages; b += 4 * PLAN) {
        const int p0 = b + 4 * t;
        int hole[4], mover[4], nh = 0, nm = 0, th, tm;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = p0 + j;
            const bool in = p < n_pages, live = in && refcount[p] > 0;
            hole[j] = in && !live && p < n_live;
            mover[j] = live && p >= n_live;
            nh += hole[j];
            nm += mover[j];
            if (in && !mover[j]) moved_to[p] = live ? p : -1;
        }
        int rh = holes + block_prefix(nh, s_sum, th), rm = movers + block_prefix(nm, s_sum, tm);
        // as many holes below n_live as live pages from it on, so 2 * movers <= n_pages
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (hole[j]) moves[2 * rh++ + 1] = p0 + j;
            if (mover[j]) moves[2 * rm++] = p0 + j;
        }
        holes += th;
        movers += tm;
    }
    __syncthreads();
    for (int r = t; r < movers; r += PLAN) {
        const int from = moves[2 * r], to = moves[2 * r + 1];
        moved_to[from] = to;
        refcount[to] = refcount[from];
        refcount[from] = 0;
    }
    if (t == 0) {
        counts[0] = n_live;
        counts[1] = movers;
    }
}

// The first `remap` workgroups rewrite the table, the others move pages.
__global__ __launch_bounds__(256) void cache_compact_move_kernel(const CachePools pools, int n_pages, int32_t *table,
                                                                 size_t entries, int remap,
                                                                 const int32_t *__restrict__ moved_to,
                                                                 const int32_t *__restrict__ moves,
                                                                 const int32_t *__restrict__ counts)
{
    const int b = (int)blockIdx.x;
    if (b < remap) {
        for (size_t e = (size_t)b * 256 + threadIdx.x; e < entries; e += (size_t)remap * 256) {
            const int p = table[e];
            if (p != -1) table[e] = p >= 0 && p < n_pages ? moved_to[p] : -1;
        }
        return;
    }
    const long work = (long)counts[1] * pools.slices;
    for (long i = b - remap; i < work; i += (long)gridDim.x - remap) {
        const int r = (int)(i / pools.slices);
        copy_slice(pools, (int)(i % pools.slices), moves[2 * r], moves[2 * r + 1], always);
    }
}

hipError_t launch_cache_copy(const CachePools &pools, int n_dst, int n_src, const int32_t *dst_pages,
                             const int32_t *src_pages, int n, hipStream_t stream)
{
    hipLaunchKernelGGL(cache_copy_kernel, dim3((unsigned)((size_t)n * pools.slices)), dim3(256), 0, stream, pools,
                       n_dst, n_src, dst_pages, src_pages, n);
    return hipGetLastError();
}

hipError_t launch_cache_fork(const CachePools &pools, int n_pages, int32_t *table, int rows, int per_row,
                             int32_t *refcount, const int32_t *parents, const int32_t *children, int n,
                             int32_t *old_pages, int32_t *new_pages, hipStream_t stream)
{
    hipLaunchKernelGGL(cache_fork_plan_kernel, dim3(1), dim3(PLAN), 0, stream, n_pages, table, rows, per_row, refcount,
                       parents, children, n, old_pages, new_pages);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || pools.slices == 0) return e;
    hipLaunchKernelGGL(cache_fork_copy_kernel, dim3((unsigned)((size_t)n * pools.slices)), dim3(256), 0, stream, pools,
                       old_pages, new_pages);
    return hipGetLastError();
}

hipError_t launch_cache_free(int32_t *table, int rows, int per_row, int32_t *refcount, int n_pages,
                             const int32_t *free_rows, int n, hipStream_t stream)
{
    const size_t blocks = ((size_t)n * per_row + 255) / 256;
    hipLaunchKernelGGL(cache_free_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream, table,
                       rows, per_row, refcount, n_pages, free_rows, n);
    return hipGetLastError();
}

hipError_t launch_cache_compact(const CachePools &pools, int n_pages, int32_t *table, int rows, int per_row,
                                int32_t *refcount, int32_t *moved_to, int32_t *moves, int32_t *counts,
                                hipStream_t stream)
{
    hipLaunchKernelGGL(cache_compact_plan_kernel, dim3(1), dim3(PLAN), 0, stream, n_pages, refcount, moved_to, moves,
                       counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t entries = (size_t)rows * per_row;
    const size_t remap = entries == 0 ? 0 : (entries + 255) / 256 < 256 ? (entries + 255) / 256 : 256;
    // the number of moves is on the device: a grid for the most there can be, up to one that fills the chip
    const size_t most = (size_t)(n_pages / 2) * pools.slices;
    const size_t grid = remap + (most < 4096 ? most : 4096);
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL(cache_compact_move_kernel, dim3((unsigned)grid), dim3(256), 0, stream, pools, n_pages, table,
                       entries, (int)remap, moved_to, moves, counts);
    return hipGetLastError();
}

}  // namespace kda

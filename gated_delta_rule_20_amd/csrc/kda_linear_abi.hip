// kda_linear_abi.hip -- the C entry points of linear attention with a decay per
// head and of the state cache's pages (include/kda.h): argument validation and
// kernel dispatch.  As in kda_abi.hip, every check runs before anything is
// enqueued, and nothing here allocates device memory or synchronises.
#include "kda.h"
#include "kda_abi.h"
#include "kda_linear.h"

using namespace kda_abi;

namespace {

bool head_dim_ok(int d) { return d == 64 || d == 128; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

kda_status_t check_heads(int dtype, int H, int Hk, int Dk, int Dv, float scale)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERROR_INVALID_VALUE, "dtype %d is not a kda_dtype_t", dtype);
    if (!head_dim_ok(Dk) || !head_dim_ok(Dv))
        return fail(KDA_ERROR_NOT_SUPPORTED, "head dims Dk=%d Dv=%d: each must be 64 or 128", Dk, Dv);
    if (H < 1 || Hk < 1 || H % Hk != 0)
        return fail(KDA_ERROR_INVALID_VALUE, "need Hk >= 1 and H a multiple of it (got H=%d Hk=%d)", H, Hk);
    if (!(scale - scale == 0.0f)) return fail(KDA_ERROR_INVALID_VALUE, "scale must be finite");
    return KDA_SUCCESS;
}

struct Ptr {
    const void *p;
    const char *name;
};

// Required device arrays: not NULL, 16-byte aligned.
kda_status_t check_required(const Ptr *a, int n)
{
    for (int i = 0; i < n; ++i) {
        if (!a[i].p) return fail(KDA_ERROR_INVALID_VALUE, "%s is NULL", a[i].name);
        if (!aligned16(a[i].p)) return fail(KDA_ERROR_INVALID_VALUE, "%s is not 16-byte aligned", a[i].name);
    }
    return KDA_SUCCESS;
}

kda_status_t check_decay(const float *g)
{
    if (!g) return fail(KDA_ERROR_INVALID_VALUE, "g is NULL");
    if (!aligned4(g)) return fail(KDA_ERROR_INVALID_VALUE, "g is not 4-byte aligned");
    return KDA_SUCCESS;
}

kda_status_t plan_pools(const kda_cache_pool_t *pools, int n, bool two, kda::CachePools *out)
{
    out->n = 0;
    out->slices = 0;
    if (n < 0 || n > KDA_CACHE_MAX_POOLS)
        return fail(KDA_ERROR_INVALID_VALUE, "n_pools=%d: must be 0..%d", n, KDA_CACHE_MAX_POOLS);
    if (n > 0 && !pools) return fail(KDA_ERROR_INVALID_VALUE, "pools is NULL");
    long long slices = 0;
    for (int i = 0; i < n; ++i) {
        if (!pools[i].dst) return fail(KDA_ERROR_INVALID_VALUE, "pool %d is NULL", i);
        if (pools[i].page_bytes < 1) return fail(KDA_ERROR_INVALID_VALUE, "pool %d has no page bytes", i);
        kda::CachePool &p = out->pool[i];
        p.dst = (char *)pools[i].dst;
        p.src = two && pools[i].src ? (const char *)pools[i].src : p.dst;
        p.page_bytes = pools[i].page_bytes;
        const uintptr_t low = (uintptr_t)p.dst | (uintptr_t)p.src | (uintptr_t)p.page_bytes;
        p.unit = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : low % 2 == 0 ? 2 : 1;
        if (p.page_bytes > ((size_t)1 << 40)) return fail(KDA_ERROR_NOT_SUPPORTED, "pool %d: pages above 1 TiB", i);
        p.slices = (int)((p.page_bytes + kda::CACHE_SLICE - 1) / kda::CACHE_SLICE);
        slices += p.slices;
    }
    if (slices > 0x7fffffffLL) return fail(KDA_ERROR_NOT_SUPPORTED, "pages too large");
    out->n = n;
    out->slices = (int)slices;
    return KDA_SUCCESS;
}

kda_status_t check_tables(int n_pages, const int32_t *table, int rows, int per_row, const int32_t *refcount)
{
    if (n_pages < 0 || n_pages > 0x3fffffff || rows < 0 || per_row < 0)
        return fail(KDA_ERROR_INVALID_VALUE, "need 0 <= n_pages < 2^30, rows >= 0, per_row >= 0 (got %d, %d, %d)", n_pages,
                    rows, per_row);
    if ((size_t)rows * per_row > 0 && !table) return fail(KDA_ERROR_INVALID_VALUE, "table is NULL");
    if (n_pages > 0 && !refcount) return fail(KDA_ERROR_INVALID_VALUE, "refcount is NULL");
    if (!aligned4(table) || !aligned4(refcount))
        return fail(KDA_ERROR_INVALID_VALUE, "table and refcount must be 4-byte aligned");
    return KDA_SUCCESS;
}

kda_status_t check_list(const int32_t *a, int n, const char *name)
{
    if (n < 0) return fail(KDA_ERROR_INVALID_VALUE, "n=%d: must be >= 0", n);
    if (n > 0 && !a) return fail(KDA_ERROR_INVALID_VALUE, "%s is NULL", name);
    if (!aligned4(a)) return fail(KDA_ERROR_INVALID_VALUE, "%s is not 4-byte aligned", name);
    return KDA_SUCCESS;
}

kda_status_t check_grid(const kda::CachePools &pools, long long pages)
{
    if (pages * (long long)pools.slices > 0x7fffffffLL)
        return fail(KDA_ERROR_NOT_SUPPORTED, "too many page bytes for one call");
    return KDA_SUCCESS;
}

}  // namespace

#define KDA_TRY(x)                              \
    do {                                        \
        const kda_status_t st_ = (x);           \
        if (st_ != KDA_SUCCESS) return st_;     \
    } while (0)

extern "C" {

kda_status_t kda_linear_recurrent_step(const kda_linear_step_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    KDA_TRY(check_heads(a->dtype, a->H, a->Hk, a->Dk, a->Dv, a->scale));
    if (a->N < 0) return fail(KDA_ERROR_INVALID_VALUE, "need N >= 0 (got N=%d)", a->N);
    if (a->n_slots < 0) return fail(KDA_ERROR_INVALID_VALUE, "need n_slots >= 0 (got %d)", a->n_slots);
    if (!a->slots && a->n_slots < a->N)
        return fail(KDA_ERROR_INVALID_VALUE, "without slots n_slots=%d must be at least N=%d", a->n_slots, a->N);
    // up to four workgroups per (sequence, head) pair, where pairs are few
    if ((long long)a->N * a->H > 0x3fffffffLL) return fail(KDA_ERROR_NOT_SUPPORTED, "N*H too large");
    if (a->N == 0) return ok();
    KDA_TRY(check_decay(a->g));
    const Ptr req[] = {{a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->state, "state"}, {a->new_state, "new_state"}, {a->o, "o"}};
    KDA_TRY(check_required(req, 6));
    if (!aligned4(a->slots)) return fail(KDA_ERROR_INVALID_VALUE, "slots is not 4-byte aligned");
    const uintptr_t x = (uintptr_t)a->state, y = (uintptr_t)a->new_state;
    const size_t bytes = (size_t)a->n_slots * a->H * a->Dk * a->Dv * 4;
    if (x != y && x < y + bytes && y < x + bytes)
        return fail(KDA_ERROR_INVALID_VALUE, "new_state overlaps state without being it");
    kda::LinearStepParams p;
    p.N = a->N; p.H = a->H; p.group = a->H / a->Hk;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.g_per_head = a->g_per_head != 0;
    p.scale = a->scale;
    p.slots = a->slots; p.n_slots = a->n_slots;
    p.state = a->state; p.new_state = a->new_state; p.o = a->o;
    const hipError_t e = kda::launch_linear_step(a->dtype == KDA_BF16, a->Dk, a->Dv, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_linear_recurrent_step launch");
    return ok();
}

kda_status_t kda_cache_copy(const kda_cache_pool_t *pools, int32_t n_pools, int32_t n_dst_pages, int32_t n_src_pages,
                            const int32_t *dst_pages, const int32_t *src_pages, int32_t n, void *stream)
{
    kda::CachePools ps;
    KDA_TRY(plan_pools(pools, n_pools, true, &ps));
    if (n_dst_pages < 0 || n_src_pages < 0)
        return fail(KDA_ERROR_INVALID_VALUE, "page counts must be >= 0 (got %d, %d)", n_dst_pages, n_src_pages);
    KDA_TRY(check_list(dst_pages, n, "dst_pages"));
    KDA_TRY(check_list(src_pages, n, "src_pages"));
    for (int i = 0; i < ps.n; ++i) {
        const uintptr_t d = (uintptr_t)ps.pool[i].dst, s = (uintptr_t)ps.pool[i].src;
        const size_t b = ps.pool[i].page_bytes;
        if (d != s && d < s + b * (size_t)n_src_pages && s < d + b * (size_t)n_dst_pages)
            return fail(KDA_ERROR_INVALID_VALUE, "pool %d: dst overlaps src without being it", i);
    }
    KDA_TRY(check_grid(ps, n));
    if (n == 0 || ps.slices == 0) return ok();
    const hipError_t e = kda::launch_cache_copy(ps, n_dst_pages, n_src_pages, dst_pages, src_pages, n, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_cache_copy launch");
    return ok();
}

kda_status_t kda_cache_fork(const kda_cache_pool_t *pools, int32_t n_pools, int32_t n_pages, int32_t *table, int32_t rows,
                            int32_t per_row, int32_t *refcount, const int32_t *parents, const int32_t *children, int32_t n,
                            int32_t *old_pages, int32_t *new_pages, void *stream)
{
    kda::CachePools ps;
    KDA_TRY(plan_pools(pools, n_pools, false, &ps));
    KDA_TRY(check_tables(n_pages, table, rows, per_row, refcount));
    KDA_TRY(check_list(parents, n, "parents"));
    KDA_TRY(check_list(children, n, "children"));
    KDA_TRY(check_list(old_pages, n, "old_pages"));
    KDA_TRY(check_list(new_pages, n, "new_pages"));
    KDA_TRY(check_grid(ps, n));
    if (n == 0) return ok();
    const hipError_t e = kda::launch_cache_fork(ps, n_pages, table, rows, per_row, refcount, parents, children, n, old_pages,
                                                new_pages, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_cache_fork launch");
    return ok();
}

kda_status_t kda_cache_free(int32_t *table, int32_t rows, int32_t per_row, int32_t *refcount, int32_t n_pages,
                            const int32_t *free_rows, int32_t n, void *stream)
{
    KDA_TRY(check_tables(n_pages, table, rows, per_row, refcount));
    KDA_TRY(check_list(free_rows, n, "free_rows"));
    if (n == 0 || rows == 0 || per_row == 0) return ok();
    const hipError_t e = kda::launch_cache_free(table, rows, per_row, refcount, n_pages, free_rows, n, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_cache_free launch");
    return ok();
}

kda_status_t kda_cache_compact(const kda_cache_pool_t *pools, int32_t n_pools, int32_t n_pages, int32_t *table, int32_t rows,
                               int32_t per_row, int32_t *refcount, int32_t *moved_to, int32_t *moves, int32_t *counts,
                               void *stream)
{
    kda::CachePools ps;
    KDA_TRY(plan_pools(pools, n_pools, false, &ps));
    KDA_TRY(check_tables(n_pages, table, rows, per_row, refcount));
    KDA_TRY(check_list(moved_to, n_pages, "moved_to"));
    KDA_TRY(check_list(moves, n_pages, "moves"));
    KDA_TRY(check_list(counts, 2, "counts"));
    const hipError_t e = kda::launch_cache_compact(ps, n_pages, table, rows, per_row, refcount, moved_to, moves, counts,
                                                   (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_cache_compact launch");
    return ok();
}

}  // extern "C"

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

bool overlap(const void *a, const void *b, size_t bytes)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + bytes && y < x + bytes;
}

kda_status_t plan_pools(const kda_cache_pool_t *pools, int n, bool two, kda::CachePools *out)
{
    *out = {};
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
        p.slices = (int)((p.page_bytes - 1) / kda::CACHE_SLICE + 1);
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

// A launch has fewer than 2^32 threads.  Checked here, so that no call is turned away after its first kernel.
bool launchable(long long workgroups, long long threads) { return workgroups <= 0xffffffffLL / threads; }

kda_status_t check_grid(const kda::CachePools &pools, long long pages)
{
    if (!launchable(pages * (long long)pools.slices, 256))
        return fail(KDA_ERROR_NOT_SUPPORTED, "too many page bytes for one call");
    return KDA_SUCCESS;
}

// Tokens per segment and what the workspace holds.  A sequence is cut only
// where its (sequence, head) pairs leave compute units idle: about SEGMENTS
// segments in all keep two workgroups on each of the 256 units.  Where even
// the shortest segments do not fill the chip, a call's time is one workgroup's:
// about 7 us for every 64 tokens of a segment, over both passes, and 0.8 us for every segment
// before its own, which is least at sqrt(7.3 * tokens) tokens (T = 1024, H = 4: 256
// tokens 31 us, 128 tokens 22 us; T = 4096, H = 8: 128, 192, 256 and 512 tokens 39, 37, 40 and 58 us, backward 96, 99, 109 and 167 us).
// Backwards one workgroup fills a unit, so segments below ANCHOR tokens are made for one
// workgroup a unit (T = 2048, H = 32: 256 tokens 124 us, with twice the segments 149 us); above, two rounds of shorter
// segments are as good (T = 8192, H = 32: 512 tokens 365 us, 1024 tokens 362 us; T = 16384: 1024 tokens 639 us, 2048 tokens 668 us).
constexpr int MIN_SEGMENT = 128, SEGMENTS = 512, ANCHOR = 512;

struct LinearPlan {
    int N, rows, seg, anchor, n_seg, n_part, n_anchors;
    bool first_pass, sum_parts;
};

struct LinearShape {
    int32_t B, T, H, Hk, Dk, Dv, dtype;
    const int32_t *cu;
    int32_t N;
    float scale;
};

kda_status_t plan_linear(const LinearShape &a, bool backward, LinearPlan *pl)
{
    const kda_status_t st = check_heads(a.dtype, a.H, a.Hk, a.Dk, a.Dv, a.scale);
    if (st != KDA_SUCCESS) return st;
    if (a.B < 1 || a.T < 0) return fail(KDA_ERROR_INVALID_VALUE, "need B >= 1, T >= 0 (got B=%d T=%d)", a.B, a.T);
    if (a.cu) {
        if (a.B != 1) return fail(KDA_ERROR_INVALID_VALUE, "cu_seqlens requires B == 1 (got B=%d)", a.B);
        if (a.N < 1) return fail(KDA_ERROR_INVALID_VALUE, "cu_seqlens requires N >= 1 (got N=%d)", a.N);
        if (!aligned4(a.cu)) return fail(KDA_ERROR_INVALID_VALUE, "cu_seqlens is not 4-byte aligned");
    }
    const long long rows = (long long)a.B * a.T;
    pl->N = a.cu ? a.N : a.B;
    if (rows > 0x7fffffffLL || (long long)pl->N * a.H > 0x0fffffffLL || a.H > (1 << 15))
        return fail(KDA_ERROR_NOT_SUPPORTED, "problem too large for 32-bit token/pair indices");
    pl->rows = (int)rows;
    long long seg = rows * a.H / SEGMENTS;
    if (seg > (1 << 28)) seg = 1 << 28;
    if (backward && seg < ANCHOR) seg = 2 * seg < ANCHOR ? 2 * seg : ANCHOR;
    // packed: the lengths are on the device; four times their mean stands for the longest
    const long long longest = a.cu && a.N > 4 ? 4 * rows / a.N : a.cu ? rows : a.T;
    while (seg < MIN_SEGMENT || seg * seg * 10 < 73 * longest) seg = seg < MIN_SEGMENT ? MIN_SEGMENT : seg + KDA_CHUNK;
    seg = (seg + KDA_CHUNK - 1) / KDA_CHUNK * KDA_CHUNK;
    if (seg > ANCHOR) seg = (seg + ANCHOR - 1) / ANCHOR * ANCHOR;
    pl->seg = (int)seg;
    pl->anchor = seg < ANCHOR ? (int)seg : ANCHOR;
    const auto over = [](int len, int by) { return len <= 0 ? 0 : (len - 1) / by; };  // pieces behind the first
    const long long n = a.cu ? rows / seg + a.N : (long long)a.B * (over(a.T, pl->seg) + 1);
    if (n * a.H > 0x7fffffffLL) return fail(KDA_ERROR_NOT_SUPPORTED, "too many segments");
    pl->n_seg = (int)n;
    pl->n_part = (int)(a.cu ? rows / seg : (long long)a.B * over(a.T, pl->seg));
    pl->n_anchors = (int)(a.cu ? rows / pl->anchor : (long long)a.B * over(a.T, pl->anchor));
    pl->first_pass = over(a.T, pl->seg) > 0;     // packed: some sequence may be that long
    // where summing them once pays: figures at linear_scan_kernel
    pl->sum_parts = backward && pl->first_pass && longest > 6 * seg && (long long)pl->N * a.H <= 16;
    return KDA_SUCCESS;
}

// One workgroup for each segment and head.
kda_status_t check_segments(const LinearPlan &pl, int H, int threads)
{
    if (!launchable((long long)pl.n_seg * H, threads))
        return fail(KDA_ERROR_NOT_SUPPORTED, "too many segments for one call: %d of %d heads, at most %lld in all", pl.n_seg, H,
                    0xffffffffLL / threads);
    return KDA_SUCCESS;
}

struct Carver {
    size_t used = 0;
    char *base;
    explicit Carver(void *b) : base((char *)b) {}
    void *take(size_t bytes)
    {
        const size_t at = used;
        used += (bytes + 255) / 256 * 256;
        return base ? base + at : nullptr;
    }
};

kda_status_t check_workspace(void *ws, size_t have, size_t need)
{
    if (need == 0) return KDA_SUCCESS;
    if (!ws) return fail(KDA_ERROR_WORKSPACE, "workspace is NULL but %zu bytes are needed", need);
    if (have < need) return fail(KDA_ERROR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    if ((uintptr_t)ws & 255u) return fail(KDA_ERROR_WORKSPACE, "workspace is not 256-byte aligned");
    return KDA_SUCCESS;
}

LinearShape shape_of(const kda_linear_fwd_args_t *a)
{
    return {a->B, a->T, a->H, a->Hk, a->Dk, a->Dv, a->dtype, a->cu_seqlens, a->N, a->scale};
}
LinearShape shape_of(const kda_linear_bwd_args_t *a)
{
    return {a->B, a->T, a->H, a->Hk, a->Dk, a->Dv, a->dtype, a->cu_seqlens, a->N, a->scale};
}

template <typename A> kda::LinearChunkParams chunk_params(const A *a, const LinearPlan &pl)
{
    kda::LinearChunkParams p = {};
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.g_per_head = a->g_per_head != 0;
    p.scale = a->scale;
    p.cu = a->cu_seqlens; p.N = pl.N; p.T = a->T; p.rows = pl.rows;
    p.H = a->H; p.group = a->H / a->Hk;
    p.seg = pl.seg; p.n_seg = pl.n_seg; p.n_part = pl.n_part;
    p.anchor_tokens = pl.anchor; p.n_anchors = pl.n_anchors;
    p.h0 = a->initial_state;
    return p;
}

void take_tables(Carver &c, const LinearPlan &pl, kda::LinearChunkParams *p)
{
    if (!p->cu || pl.N <= kda::TABLE_SEQUENCES) return;
    p->seq_of = (int32_t *)c.take(sizeof(int32_t) * (size_t)pl.n_seg);
    p->first_seg = (int32_t *)c.take(sizeof(int32_t) * (size_t)pl.N);
    p->first_anchor = (int32_t *)c.take(sizeof(int32_t) * (size_t)pl.N);
}

// The first pass's buffers.
void take_parts(Carver &c, const LinearPlan &pl, int H, size_t state, float **part, float **dec)
{
    *part = (float *)c.take(state * pl.n_part);
    *dec = (float *)c.take(sizeof(float) * (size_t)H * pl.n_part);
}

size_t plan_fwd(const kda_linear_fwd_args_t *a, const LinearPlan &pl, void *ws, kda::LinearChunkParams *p)
{
    Carver c(ws);
    *p = chunk_params(a, pl);
    p->hT = a->final_state;
    p->o = a->o;
    p->ckpt = a->checkpoints;
    p->ckpt_every = a->checkpoint_every;
    p->ckpt_slots = a->checkpoint_slots;
    take_tables(c, pl, p);
    const size_t state = sizeof(float) * a->H * a->Dk * a->Dv;
    if (pl.first_pass) {
        take_parts(c, pl, a->H, state, &p->part, &p->dec);
        p->defer = overlap(a->initial_state, a->final_state, state * pl.N);
    }
    return c.used;
}

size_t plan_bwd(const kda_linear_bwd_args_t *a, const LinearPlan &pl, void *ws, kda::LinearBwdParams *b)
{
    Carver c(ws);
    *b = {};
    b->c = chunk_params(a, pl);
    b->d_o = a->d_o; b->dhT = a->d_final_state; b->dh0 = a->d_initial_state;
    b->dq = a->dq; b->dk = a->dk; b->dv = a->dv; b->dg = a->dg;
    take_tables(c, pl, &b->c);
    const size_t state = sizeof(float) * a->H * a->Dk * a->Dv;
    if (pl.first_pass) {
        take_parts(c, pl, a->H, state, &b->c.part, &b->c.dec);
        b->c.defer = overlap(a->d_final_state, a->d_initial_state, state * pl.N);
        take_parts(c, pl, a->H, state, &b->part_fwd, &b->dec_fwd);
        b->c.part_tr = (float *)c.take(state * pl.n_part);
        if (pl.sum_parts) {
            b->c.summed = 1;
            b->sum_fwd = (float *)c.take(sizeof(float) * (size_t)a->H * pl.n_part);
            b->sum_rev = (float *)c.take(sizeof(float) * (size_t)a->H * pl.n_part);
        }
    }
    if (a->dg) {
        b->c.y = (float *)c.take(sizeof(float) * (size_t)a->H * pl.rows);
        b->c.anchor_end = a->d_final_state != nullptr;
        b->c.anchors = (float *)c.take(state * ((size_t)pl.n_anchors + (b->c.anchor_end ? pl.N : 0)));
        if (a->g_per_head) b->dg_part = (double *)c.take(sizeof(double) * (size_t)a->H * pl.n_seg);
    }
    if (a->H != a->Hk) {
        const size_t bytes = sizeof(float) * (size_t)pl.rows * a->H * a->Dk;
        b->c.wide = 1;
        b->dq_out = a->dq; b->dk_out = a->dk;
        b->dq = c.take(bytes);
        b->dk = c.take(bytes);
    }
    return c.used;
}

}  // namespace

#define KDA_TRY(x)                              \
    do {                                        \
        const kda_status_t st_ = (x);           \
        if (st_ != KDA_SUCCESS) return st_;     \
    } while (0)

extern "C" {

kda_status_t kda_linear_chunk_fwd_workspace_size(const kda_linear_fwd_args_t *a, size_t *bytes)
{
    if (!a || !bytes) return fail(KDA_ERROR_INVALID_VALUE, "args or bytes is NULL");
    LinearPlan pl;
    KDA_TRY(plan_linear(shape_of(a), false, &pl));
    kda::LinearChunkParams p;
    *bytes = plan_fwd(a, pl, nullptr, &p);
    return ok();
}

kda_status_t kda_linear_chunk_fwd(const kda_linear_fwd_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    LinearPlan pl;
    KDA_TRY(plan_linear(shape_of(a), false, &pl));
    KDA_TRY(check_segments(pl, a->H, kda::LINEAR_FWD_THREADS));
    if (pl.rows > 0) {
        KDA_TRY(check_decay(a->g));
        const Ptr req[] = {{a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->o, "o"}};
        KDA_TRY(check_required(req, 4));
    }
    if (!aligned16(a->initial_state)) return fail(KDA_ERROR_INVALID_VALUE, "initial_state is not 16-byte aligned");
    if (!aligned16(a->final_state)) return fail(KDA_ERROR_INVALID_VALUE, "final_state is not 16-byte aligned");
    if (a->checkpoints) {
        if (!aligned16(a->checkpoints)) return fail(KDA_ERROR_INVALID_VALUE, "checkpoints is not 16-byte aligned");
        if (a->checkpoint_every < 1 || a->checkpoint_slots < 1 || a->checkpoint_every > 0x1ffffff)
            return fail(KDA_ERROR_INVALID_VALUE, "need 1 <= checkpoint_every < 2^25 and checkpoint_slots >= 1 (got %d, %d)",
                        a->checkpoint_every, a->checkpoint_slots);
    }
    kda::LinearChunkParams p;
    KDA_TRY(check_workspace(a->workspace, a->workspace_bytes, plan_fwd(a, pl, a->workspace, &p)));
    if (pl.rows == 0 && !a->final_state) return ok();
    const hipError_t e = kda::launch_linear_fwd(a->dtype == KDA_BF16, a->Dk, a->Dv, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_linear_chunk_fwd launch");
    return ok();
}

kda_status_t kda_linear_chunk_bwd_workspace_size(const kda_linear_bwd_args_t *a, size_t *bytes)
{
    if (!a || !bytes) return fail(KDA_ERROR_INVALID_VALUE, "args or bytes is NULL");
    LinearPlan pl;
    KDA_TRY(plan_linear(shape_of(a), true, &pl));
    kda::LinearBwdParams b;
    *bytes = plan_bwd(a, pl, nullptr, &b);
    return ok();
}

kda_status_t kda_linear_chunk_bwd(const kda_linear_bwd_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    LinearPlan pl;
    KDA_TRY(plan_linear(shape_of(a), true, &pl));
    KDA_TRY(check_segments(pl, a->H, kda::LINEAR_BWD_THREADS));
    if (pl.rows > 0) {
        KDA_TRY(check_decay(a->g));
        const Ptr req[] = {{a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->d_o, "d_o"}, {a->dq, "dq"}, {a->dk, "dk"}, {a->dv, "dv"}};
        KDA_TRY(check_required(req, 7));
    }
    if (!aligned4(a->dg)) return fail(KDA_ERROR_INVALID_VALUE, "dg is not 4-byte aligned");
    if (!aligned16(a->initial_state)) return fail(KDA_ERROR_INVALID_VALUE, "initial_state is not 16-byte aligned");
    if (!aligned16(a->d_final_state)) return fail(KDA_ERROR_INVALID_VALUE, "d_final_state is not 16-byte aligned");
    if (!aligned16(a->d_initial_state)) return fail(KDA_ERROR_INVALID_VALUE, "d_initial_state is not 16-byte aligned");
    kda::LinearBwdParams b;
    KDA_TRY(check_workspace(a->workspace, a->workspace_bytes, plan_bwd(a, pl, a->workspace, &b)));
    if (pl.rows == 0 && !a->d_initial_state && !(a->dg && a->g_per_head)) return ok();
    const hipError_t e = kda::launch_linear_bwd(a->dtype == KDA_BF16, a->Dk, a->Dv, b, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_linear_chunk_bwd launch");
    return ok();
}

kda_status_t kda_linear_recurrent_step(const kda_linear_step_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    KDA_TRY(check_heads(a->dtype, a->H, a->Hk, a->Dk, a->Dv, a->scale));
    if (a->N < 0) return fail(KDA_ERROR_INVALID_VALUE, "need N >= 0 (got N=%d)", a->N);
    if (a->n_slots < 0) return fail(KDA_ERROR_INVALID_VALUE, "need n_slots >= 0 (got %d)", a->n_slots);
    if (!a->slots && a->n_slots < a->N)
        return fail(KDA_ERROR_INVALID_VALUE, "without slots n_slots=%d must be at least N=%d", a->n_slots, a->N);
    // one workgroup of 256 threads per (sequence, head) pair (more where pairs are few)
    if (!launchable((long long)a->N * a->H, 256)) return fail(KDA_ERROR_NOT_SUPPORTED, "N*H too large");
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

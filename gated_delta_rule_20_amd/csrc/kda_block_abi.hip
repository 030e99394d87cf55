// kda_block_abi.hip -- the C entry points of the gated scan, the norms around a
// block and 8-bit activations (include/kda.h): argument validation and kernel
// dispatch.  Every check runs before anything is enqueued, and nothing here
// allocates device memory or synchronises.
#include "kda.h"
#include "kda_abi.h"
#include "kda_block.h"

using namespace kda_abi;

#define KDA_TRY(x)                              \
    do {                                        \
        const kda_status_t st_ = (x);           \
        if (st_ != KDA_SUCCESS) return st_;     \
    } while (0)

namespace {

int element_bytes(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }
bool launchable(long long workgroups, long long threads) { return workgroups <= 0xffffffffLL / threads; }

kda_status_t check_dtype(int dtype, const char *name)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERROR_INVALID_VALUE, "%s %d is not a kda_dtype_t", name, dtype);
    return KDA_SUCCESS;
}

// A call's type and a second one that is the same or float32.
kda_status_t check_dtypes(int dtype, int other, const char *name)
{
    KDA_TRY(check_dtype(dtype, "dtype"));
    KDA_TRY(check_dtype(other, name));
    if (dtype == KDA_F32 && other != KDA_F32)
        return fail(KDA_ERROR_NOT_SUPPORTED, "%s must be float32 in a float32 call", name);
    return KDA_SUCCESS;
}

kda_status_t check_array(const void *p, int bytes, const char *name)
{
    if ((uintptr_t)p % (unsigned)bytes) return fail(KDA_ERROR_INVALID_VALUE, "%s is not %d-byte aligned", name, bytes);
    return KDA_SUCCESS;
}

kda_status_t check_given(const void *p, int bytes, const char *name)
{
    if (!p) return fail(KDA_ERROR_INVALID_VALUE, "%s is NULL", name);
    return check_array(p, bytes, name);
}

kda_status_t check_stride(int64_t stride, int C, const char *name)
{
    if (stride < C || stride > (1 << 24))
        return fail(KDA_ERROR_INVALID_VALUE, "%s=%lld: must be %d (the row) to 2^24", name, (long long)stride, C);
    return KDA_SUCCESS;
}

// Rows that are elements or, with scales, codes (any address, dense).
kda_status_t check_rows(const void *p, const float *scales, int bytes, const char *name)
{
    KDA_TRY(check_given(p, scales ? 1 : bytes, name));
    return check_array(scales, 4, "scales");
}

kda_status_t check_packed(const void *codes, const float *scales, const char *name)
{
    if (!codes != !scales) return fail(KDA_ERROR_INVALID_VALUE, "%s: codes and scales come together", name);
    return check_array(scales, 4, name);
}

bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + b_bytes && y < x + a_bytes;
}

kda_status_t check_workspace(void *ws, size_t have, size_t need)
{
    if (need == 0) return KDA_SUCCESS;
    if (!ws) return fail(KDA_ERROR_WORKSPACE, "workspace is NULL but %zu bytes are needed", need);
    if (have < need) return fail(KDA_ERROR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    if ((uintptr_t)ws & 255u) return fail(KDA_ERROR_WORKSPACE, "workspace is not 256-byte aligned");
    return KDA_SUCCESS;
}

// ---- gated scan ------------------------------------------------------------------

kda_status_t check_decay(int C, const float *A_log, float g_min)
{
    if (C < 1 || C > (1 << 24)) return fail(KDA_ERROR_INVALID_VALUE, "need 1 <= C <= 2^24 (got %d)", C);
    KDA_TRY(check_array(A_log, 4, "A_log"));
    if (A_log && !(g_min < 0.f && g_min >= -1e6f))
        return fail(KDA_ERROR_INVALID_VALUE, "g_min must be below 0 and -1e6 at least (got %g)", (double)g_min);
    return KDA_SUCCESS;
}

template <typename A> kda_status_t plan_scan(const A *a, kda::ScanParams *p)
{
    *p = {};
    KDA_TRY(check_dtypes(a->dtype, a->g_dtype, "g_dtype"));
    KDA_TRY(check_decay(a->C, a->A_log, a->g_min));
    if (a->B < 1 || a->T < 0) return fail(KDA_ERROR_INVALID_VALUE, "need B >= 1, T >= 0 (got B=%d T=%d)", a->B, a->T);
    if (a->cu_seqlens) {
        if (a->B != 1) return fail(KDA_ERROR_INVALID_VALUE, "cu_seqlens requires B == 1 (got B=%d)", a->B);
        if (a->N < 1) return fail(KDA_ERROR_INVALID_VALUE, "cu_seqlens requires N >= 1 (got N=%d)", a->N);
        KDA_TRY(check_array(a->cu_seqlens, 4, "cu_seqlens"));
    }
    p->N = a->cu_seqlens ? a->N : a->B;
    const long long rows = (long long)a->B * a->T;
    if (rows > 0x7fffff00LL) return fail(KDA_ERROR_NOT_SUPPORTED, "too many tokens for 32-bit indices");
    // one workgroup for each segment of rows and of channels
    const long long wide = (a->C + kda::SCAN_CHANNELS - 1) / kda::SCAN_CHANNELS;
    if (!launchable((rows / kda::SCAN_ROWS + 1) * wide, 256) || p->N > (1 << 28))
        return fail(KDA_ERROR_NOT_SUPPORTED, "rows * C too large for one call");
    p->rows = (int)rows;
    p->T = a->T;
    p->C = a->C;
    p->cu = a->cu_seqlens;
    p->A_log = a->A_log;
    p->g_min = a->g_min;
    p->complement = a->complement != 0;
    p->h0 = a->initial_state;
    p->g = {a->g, nullptr, a->g_stride};
    if (rows > 0) {
        KDA_TRY(check_given(a->g, element_bytes(a->g_dtype), "g"));
        KDA_TRY(check_stride(a->g_stride, a->C, "g_stride"));
    }
    return check_array(a->initial_state, 4, "initial_state");
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

// The hand-over between segments, and the entering states' copy where the resulting ones overwrite them.
void plan_chain(Carver &c, const float *from, const float *to, kda::ScanParams *p)
{
    kda::ScanChain &k = p->chain;
    const size_t C = (size_t)p->C, states = (size_t)p->N * C;
    k.segments = p->rows > 0 ? (p->rows - 1) / kda::SCAN_ROWS + 1 : 1;
    if (k.segments > 1) {
        const size_t parts = (size_t)k.segments * C, blocks = (size_t)(k.segments / kda::SCAN_BLOCK) * C;
        const size_t whole = (size_t)(k.segments / (kda::SCAN_BLOCK * kda::SCAN_BLOCK)) * C;
        k.words = parts + blocks + whole;
        k.counters = (C + kda::SCAN_CHANNELS - 1) / kda::SCAN_CHANNELS * kda::SCAN_TICKET_STEP + 1;
        k.part = (uint64_t *)c.take(8 * k.words);
        k.blocks = k.part + parts;
        k.whole = k.blocks + blocks;
        k.tickets = (uint32_t *)c.take(4 * k.counters);
        k.gave_up = k.tickets + k.counters - 1;
    }
    if (overlap(from, 4 * states, to, 4 * states)) p->state_copy = (float *)c.take(4 * states);
}

size_t plan_scan_fwd(const kda_gated_scan_fwd_args_t *a, kda::ScanParams *p)
{
    Carver c(a->workspace);
    plan_chain(c, a->initial_state, a->final_state, p);
    return c.used;
}

size_t plan_scan_bwd(const kda_gated_scan_bwd_args_t *a, kda::ScanParams *p)
{
    Carver c(a->workspace);
    plan_chain(c, a->d_final_state, a->d_initial_state, p);
    if (a->dA_log) p->dA_part = (float *)c.take(sizeof(float) * (size_t)p->chain.segments * p->C);
    return c.used;
}

// ---- block norms -----------------------------------------------------------------

template <typename A> kda_status_t plan_norm(const A *a, kda::NormParams *p)
{
    *p = {};
    KDA_TRY(check_dtypes(a->dtype, a->x_dtype, "x_dtype"));
    if (a->R < 0) return fail(KDA_ERROR_INVALID_VALUE, "need R >= 0 (got %d)", a->R);
    if (a->R > 0x7fff0000) return fail(KDA_ERROR_NOT_SUPPORTED, "too many rows for 32-bit indices");
    if (a->D < 1) return fail(KDA_ERROR_INVALID_VALUE, "need D >= 1 (got %d)", a->D);
    if (a->D > kda::NORM_MAX_D) return fail(KDA_ERROR_NOT_SUPPORTED, "D=%d: at most %d", a->D, kda::NORM_MAX_D);
    if (!(a->eps >= 0.f)) return fail(KDA_ERROR_INVALID_VALUE, "eps must be >= 0");
    if (!(a->scale - a->scale == 0.f)) return fail(KDA_ERROR_INVALID_VALUE, "scale must be finite");
    if (a->R > 0 && !a->y && (a->gate || a->post_weight || a->res_scale))
        return fail(KDA_ERROR_INVALID_VALUE, "gate, post_weight and res_scale belong to y, which is NULL");
    p->R = a->R;
    p->D = a->D;
    p->scale = a->scale;
    p->eps = a->eps;
    p->post = a->post_weight;
    p->res = a->res_scale;
    p->pre = a->pre_weight;
    KDA_TRY(check_array(a->post_weight, 4, "post_weight"));
    KDA_TRY(check_array(a->res_scale, 4, "res_scale"));
    KDA_TRY(check_array(a->pre_weight, 4, "pre_weight"));
    return KDA_SUCCESS;
}

// Workgroups of the gradients, each with float32 sums of its own of the weights' gradients: four rows a side at least, 16 waves (of columns:
// 32) on each of 256 units at most, or as many times these as leave no side more than NORM_CHAIN rows, so that what the sums may be off by
// does not grow with the rows: 65536 x 4096 1006 us, with 256 rows in a sum (equal rows off by 64 roundings instead of 16) 967; 2^20 x 256
// 916 and 905.
// (One row at least: 256 x 4096 23.5 us either way, with four times the sums; 16: 42.5.)
void norm_parts(int R, int D, bool columns, kda::NormParams *p)
{
    const int side = kda::norm_rows(D), rows = 4 * side;
    const int most = columns ? 256 * 8 / ((D + kda::NORM_COLUMN - 1) / kda::NORM_COLUMN) : 256 * 16 / kda::norm_waves(D);
    const int n = R / rows + (R % rows != 0);
    p->groups = p->parts = n < most ? n : most;
    const int turn = most * side * kda::NORM_CHAIN;        // rows (2^18 at most)
    if (R > turn) p->parts = most * (R / turn + (R % turn != 0));
}

kda_status_t plan_norm_bwd(const kda_block_norm_bwd_args_t *a, kda::NormParams *p, size_t *bytes)
{
    const bool columns = a->D > kda::norm_row_d(a->dtype == KDA_F32);
    norm_parts(a->R, a->D, columns, p);
    const long long wide = columns ? (a->D + kda::NORM_COLUMN - 1) / kda::NORM_COLUMN : 1;
    if (!launchable(p->parts * wide, columns ? 256 : 64 * kda::norm_waves(a->D)))
        return fail(KDA_ERROR_NOT_SUPPORTED, "R * D too large for one call");
    Carver c(a->workspace);
    if (a->d_post_weight || a->d_res_scale || a->d_pre_weight) p->part = (float *)c.take(sizeof(float) * 3 * (size_t)p->parts * a->D);
    if (columns) p->numbers = (decltype(p->numbers))c.take(16 * (size_t)a->R);
    *bytes = c.used;
    return KDA_SUCCESS;
}

}  // namespace

extern "C" {

kda_status_t kda_gated_scan_fwd_workspace_size(const kda_gated_scan_fwd_args_t *a, size_t *bytes)
{
    if (!a || !bytes) return fail(KDA_ERROR_INVALID_VALUE, "args or bytes is NULL");
    kda_gated_scan_fwd_args_t b = *a;
    b.g = (const void *)16;                    // only sizes count
    b.g_stride = b.C;
    kda::ScanParams p;
    KDA_TRY(plan_scan(&b, &p));
    *bytes = plan_scan_fwd(&b, &p);
    return ok();
}

kda_status_t kda_gated_scan_fwd(const kda_gated_scan_fwd_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    kda::ScanParams p;
    KDA_TRY(plan_scan(a, &p));
    const int size = element_bytes(a->dtype);
    if (p.rows > 0) {
        KDA_TRY(check_given(a->x, size, "x"));
        KDA_TRY(check_stride(a->x_stride, a->C, "x_stride"));
        KDA_TRY(check_given(a->h, size, "h"));
    }
    KDA_TRY(check_array(a->final_state, 4, "final_state"));
    KDA_TRY(check_packed(a->h_codes, a->h_scales, "h"));
    p.x = {a->x, nullptr, a->x_stride};
    p.h = a->h;
    p.hT = a->final_state;
    p.h8 = {a->h_codes, a->h_scales};
    KDA_TRY(check_workspace(a->workspace, a->workspace_bytes, plan_scan_fwd(a, &p)));
    if (p.rows == 0 && !p.hT) return ok();
    const hipError_t e = kda::launch_scan_fwd(a->dtype == KDA_BF16, a->g_dtype == KDA_BF16, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_gated_scan_fwd launch");
    return ok();
}

kda_status_t kda_gated_scan_bwd_workspace_size(const kda_gated_scan_bwd_args_t *a, size_t *bytes)
{
    if (!a || !bytes) return fail(KDA_ERROR_INVALID_VALUE, "args or bytes is NULL");
    kda_gated_scan_bwd_args_t b = *a;
    b.g = (const void *)16;
    b.g_stride = b.C;
    kda::ScanParams p;
    KDA_TRY(plan_scan(&b, &p));
    *bytes = plan_scan_bwd(&b, &p);
    return ok();
}

kda_status_t kda_gated_scan_bwd(const kda_gated_scan_bwd_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    kda::ScanParams p;
    KDA_TRY(plan_scan(a, &p));
    const int size = element_bytes(a->dtype);
    if (a->dA_log && (!a->A_log || (!a->dg && p.rows > 0)))
        return fail(KDA_ERROR_INVALID_VALUE, "dA_log needs A_log and dg");
    if (p.rows > 0) {
        KDA_TRY(check_given(a->d_h, size, "d_h"));
        KDA_TRY(check_given(a->dx, size, "dx"));
        KDA_TRY(check_stride(a->dx_stride, a->C, "dx_stride"));
        if (a->dg) {
            KDA_TRY(check_rows(a->h, a->h_scales, size, "h"));
            KDA_TRY(check_array(a->dg, element_bytes(a->g_dtype), "dg"));
            KDA_TRY(check_stride(a->dg_stride, a->C, "dg_stride"));
            if (a->complement) {
                KDA_TRY(check_rows(a->x, a->x_scales, size, "x"));
                if (!a->x_scales) KDA_TRY(check_stride(a->x_stride, a->C, "x_stride"));
            }
        }
    }
    KDA_TRY(check_array(a->dA_log, 4, "dA_log"));
    KDA_TRY(check_array(a->d_final_state, 4, "d_final_state"));
    KDA_TRY(check_array(a->d_initial_state, 4, "d_initial_state"));
    p.x = {a->x, a->x_scales, a->x_scales ? a->C : a->x_stride};
    p.hs = {a->h, a->h_scales, a->C};
    p.d_h = a->d_h;
    p.dhT = a->d_final_state;
    p.dx = a->dx;
    p.dx_stride = a->dx_stride;
    p.dg = a->dg;
    p.dg_stride = a->dg_stride;
    p.dA = a->dA_log;
    p.dh0 = a->d_initial_state;
    KDA_TRY(check_workspace(a->workspace, a->workspace_bytes, plan_scan_bwd(a, &p)));
    if (p.rows == 0 && !p.dh0 && !p.dA) return ok();
    const hipError_t e = kda::launch_scan_bwd(a->dtype == KDA_BF16, a->g_dtype == KDA_BF16, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_gated_scan_bwd launch");
    return ok();
}

kda_status_t kda_gated_scan_step(const kda_gated_scan_step_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    KDA_TRY(check_dtypes(a->dtype, a->g_dtype, "g_dtype"));
    KDA_TRY(check_decay(a->C, a->A_log, a->g_min));
    if (a->N < 0) return fail(KDA_ERROR_INVALID_VALUE, "need N >= 0 (got N=%d)", a->N);
    if (a->n_slots < 0) return fail(KDA_ERROR_INVALID_VALUE, "need n_slots >= 0 (got %d)", a->n_slots);
    if (!a->slots && a->n_slots < a->N)
        return fail(KDA_ERROR_INVALID_VALUE, "without slots n_slots=%d must be at least N=%d", a->n_slots, a->N);
    if (!launchable((long long)a->N * ((a->C + 511) / 512), 256)) return fail(KDA_ERROR_NOT_SUPPORTED, "N * C too large");
    if (a->N == 0) return ok();
    const int size = element_bytes(a->dtype);
    KDA_TRY(check_given(a->x, size, "x"));
    KDA_TRY(check_given(a->g, element_bytes(a->g_dtype), "g"));
    KDA_TRY(check_stride(a->x_stride, a->C, "x_stride"));
    KDA_TRY(check_stride(a->g_stride, a->C, "g_stride"));
    KDA_TRY(check_given(a->state, 4, "state"));
    KDA_TRY(check_given(a->new_state, 4, "new_state"));
    KDA_TRY(check_given(a->h, size, "h"));
    KDA_TRY(check_array(a->slots, 4, "slots"));
    const size_t bytes = (size_t)a->n_slots * a->C * 4;
    if (a->state != a->new_state && overlap(a->state, bytes, a->new_state, bytes))
        return fail(KDA_ERROR_INVALID_VALUE, "new_state overlaps state without being it");
    kda::ScanStepParams p = {};
    p.N = a->N; p.C = a->C;
    p.x = {a->x, nullptr, a->x_stride};
    p.g = {a->g, nullptr, a->g_stride};
    p.A_log = a->A_log; p.g_min = a->g_min; p.complement = a->complement != 0;
    p.slots = a->slots; p.n_slots = a->n_slots;
    p.state = a->state; p.new_state = a->new_state; p.h = a->h;
    const hipError_t e = kda::launch_scan_step(a->dtype == KDA_BF16, a->g_dtype == KDA_BF16, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_gated_scan_step launch");
    return ok();
}

kda_status_t kda_block_norm_fwd(const kda_block_norm_fwd_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    kda::NormParams p;
    KDA_TRY(plan_norm(a, &p));
    if (a->R == 0) return ok();
    if (!a->y && !a->pre_weight) return fail(KDA_ERROR_INVALID_VALUE, "neither y nor pre_weight is given: nothing to compute");
    const int size = element_bytes(a->dtype), x_size = element_bytes(a->x_dtype);
    KDA_TRY(check_packed(a->x_codes, a->x_scales, "x"));
    KDA_TRY(check_packed(a->y_codes, a->y_scales, "y"));
    KDA_TRY(check_packed(a->gate_codes, a->gate_scales, "gate"));
    if ((a->y_codes && !a->y) || (a->gate_codes && !a->gate))
        return fail(KDA_ERROR_INVALID_VALUE, "codes of y or gate without it");
    KDA_TRY(check_given(a->x, x_size, "x"));
    if (a->y) {
        KDA_TRY(check_array(a->y, size, "y"));
        KDA_TRY(check_stride(a->y_stride, a->D, "y_stride"));
        KDA_TRY(check_given(a->x_out, x_size, "x_out"));
        const size_t bytes = (size_t)a->R * a->D * x_size;
        if (a->x_out != a->x && overlap(a->x_out, bytes, a->x, bytes))
            return fail(KDA_ERROR_INVALID_VALUE, "x_out overlaps x without being it");
    }
    if (a->gate) {
        KDA_TRY(check_array(a->gate, size, "gate"));
        KDA_TRY(check_stride(a->gate_stride, a->D, "gate_stride"));
    }
    if (a->pre_weight) KDA_TRY(check_given(a->n, size, "n"));
    p.x = {a->x, nullptr, a->D};
    p.y = {a->y, nullptr, a->y_stride};
    p.gate = {a->gate, nullptr, a->gate_stride};
    p.x_out = a->x_out;
    p.n = a->n;
    p.x8 = {a->x_codes, a->x_scales};
    p.y8 = {a->y_codes, a->y_scales};
    p.gate8 = {a->gate_codes, a->gate_scales};
    const hipError_t e = kda::launch_norm_fwd(a->dtype == KDA_BF16, a->x_dtype == KDA_BF16, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_block_norm_fwd launch");
    return ok();
}

kda_status_t kda_block_norm_bwd_workspace_size(const kda_block_norm_bwd_args_t *a, size_t *bytes)
{
    if (!a || !bytes) return fail(KDA_ERROR_INVALID_VALUE, "args or bytes is NULL");
    kda::NormParams p;
    KDA_TRY(plan_norm(a, &p));
    KDA_TRY(plan_norm_bwd(a, &p, bytes));
    return ok();
}

kda_status_t kda_block_norm_bwd(const kda_block_norm_bwd_args_t *a, void *stream)
{
    if (!a) return fail(KDA_ERROR_INVALID_VALUE, "args is NULL");
    kda::NormParams p;
    KDA_TRY(plan_norm(a, &p));
    const int size = element_bytes(a->dtype), x_size = element_bytes(a->x_dtype);
    if ((a->d_post_weight && !a->post_weight) || (a->d_res_scale && !a->res_scale) || (a->d_pre_weight && !a->pre_weight))
        return fail(KDA_ERROR_INVALID_VALUE, "a weight's gradient without the weight");
    if (a->R > 0 && !a->d_x_new && !a->d_n) return fail(KDA_ERROR_INVALID_VALUE, "neither d_x_new nor d_n is given");
    if (a->d_n && !a->pre_weight) return fail(KDA_ERROR_INVALID_VALUE, "d_n without pre_weight");
    if (a->R > 0) {
        KDA_TRY(check_given(a->dx, x_size, "dx"));
        KDA_TRY(check_array(a->d_x_new, x_size, "d_x_new"));
        KDA_TRY(check_array(a->d_n, size, "d_n"));
        if (a->d_n) KDA_TRY(check_rows(a->x_new, a->x_scales, x_size, "x_new"));
        const size_t bytes = (size_t)a->R * a->D * x_size;
        if (a->dx != a->d_x_new && overlap(a->dx, bytes, a->d_x_new, bytes))
            return fail(KDA_ERROR_INVALID_VALUE, "dx overlaps d_x_new without being it");
        if (a->y) {
            KDA_TRY(check_rows(a->y, a->y_scales, size, "y"));
            if (!a->y_scales) KDA_TRY(check_stride(a->y_stride, a->D, "y_stride"));
            KDA_TRY(check_given(a->dy, size, "dy"));
            KDA_TRY(check_stride(a->dy_stride, a->D, "dy_stride"));
        }
        if (a->gate) {
            KDA_TRY(check_rows(a->gate, a->gate_scales, size, "gate"));
            if (!a->gate_scales) KDA_TRY(check_stride(a->gate_stride, a->D, "gate_stride"));
            KDA_TRY(check_given(a->dgate, size, "dgate"));
            KDA_TRY(check_stride(a->dgate_stride, a->D, "dgate_stride"));
        }
    }
    KDA_TRY(check_array(a->d_post_weight, 4, "d_post_weight"));
    KDA_TRY(check_array(a->d_res_scale, 4, "d_res_scale"));
    KDA_TRY(check_array(a->d_pre_weight, 4, "d_pre_weight"));
    p.x = {a->x_new, a->x_scales, a->D};
    p.y = {a->y, a->y_scales, a->y_scales ? a->D : a->y_stride};
    p.gate = {a->gate, a->gate_scales, a->gate_scales ? a->D : a->gate_stride};
    p.d_x = a->d_x_new;
    p.d_n = a->d_n;
    p.dx = a->dx;
    p.dy = a->dy;
    p.dgate = a->dgate;
    p.dy_stride = a->dy_stride;
    p.dgate_stride = a->dgate_stride;
    p.dpost = a->d_post_weight;
    p.dres = a->d_res_scale;
    p.dpre = a->d_pre_weight;
    size_t need = 0;
    KDA_TRY(plan_norm_bwd(a, &p, &need));
    KDA_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    if (p.R == 0 && !p.dpost && !p.dres && !p.dpre) return ok();
    const hipError_t e = kda::launch_norm_bwd(a->dtype == KDA_BF16, a->x_dtype == KDA_BF16, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_block_norm_bwd launch");
    return ok();
}

static kda_status_t check_act(int dtype, int64_t R, int32_t D)
{
    KDA_TRY(check_dtype(dtype, "dtype"));
    if (R < 0 || D < 1) return fail(KDA_ERROR_INVALID_VALUE, "need R >= 0 and D >= 1 (got %lld, %d)", (long long)R, D);
    // channels are indexed in 32 bits, and R * per below stays within 64
    if (D > (1 << 24)) return fail(KDA_ERROR_NOT_SUPPORTED, "D=%d: at most 2^24", D);
    // one workgroup packs 16 groups
    const int64_t per = ((int64_t)D + kda::ACT_GROUP - 1) / kda::ACT_GROUP;
    if (R > ((int64_t)1 << 40) || !launchable((R * per + 15) / 16, 256)) return fail(KDA_ERROR_NOT_SUPPORTED, "R * D too large for one call");
    return KDA_SUCCESS;
}

kda_status_t kda_act_pack(int32_t dtype, const void *x, int64_t x_stride, int64_t R, int32_t D, int8_t *codes, float *scales,
                          void *stream)
{
    KDA_TRY(check_act(dtype, R, D));
    if (R == 0) return ok();
    KDA_TRY(check_given(x, element_bytes(dtype), "x"));
    KDA_TRY(check_stride(x_stride, D, "x_stride"));
    KDA_TRY(check_given(codes, 1, "codes"));
    KDA_TRY(check_given(scales, 4, "scales"));
    const hipError_t e = kda::launch_act_pack(dtype == KDA_BF16, {x, nullptr, x_stride}, R, D, {codes, scales}, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_act_pack launch");
    return ok();
}

kda_status_t kda_act_unpack(int32_t dtype, const int8_t *codes, const float *scales, int64_t R, int32_t D, void *x, void *stream)
{
    KDA_TRY(check_act(dtype, R, D));
    if (R == 0) return ok();
    KDA_TRY(check_given(codes, 1, "codes"));
    KDA_TRY(check_given(scales, 4, "scales"));
    KDA_TRY(check_given(x, element_bytes(dtype), "x"));
    const hipError_t e = kda::launch_act_unpack(dtype == KDA_BF16, {codes, scales, D}, R, D, x, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "kda_act_unpack launch");
    return ok();
}

}  // extern "C"

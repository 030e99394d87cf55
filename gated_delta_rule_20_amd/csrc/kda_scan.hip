// kda_scan.hip -- the gated scan  h_t = a_t h_{t-1} + m_t x_t  per channel:
// whole sequences, their gradients, one token.
#include "kda_block_dev.h"

namespace kda {

// Rows [lo, hi) of sequence s.
__device__ __forceinline__ void sequence_of(const ScanParams &p, int s, int *lo, int *hi)
{
    if (!p.cu) {
        *lo = s * p.T;
        *hi = *lo + p.T;
        return;
    }
    *lo = min(max(p.cu[s], 0), p.rows);
    *hi = min(max(p.cu[s + 1], *lo), p.rows);
}

// ---- segments --------------------------------------------------------------------
//
// h_t = a_t h_{t-1} + b_t is associative: a run of tokens maps the state before
// it to (product of a) h + (state from zero).  A workgroup takes 64 rows of
// 128 channels: 32 lanes hold 4 channels each, 8 groups of lanes 8 rows each.
// A lane runs over its rows from zero (keeping the decays), 128 threads join
// the 8 runs of a channel through LDS, and with the state before it each lane
// runs over its rows again from registers: x and g are read once, h written
// once.
//
// Segments of a call's packed rows are joined in one pass.  Workgroups take
// tickets (so a segment's predecessors run or have run already), publish what
// their rows do to a state before waiting for anything, and wait for the pairs of the segments before
// them, back to the nearest one whose last row's state is published whole
// (every `group`-th).  The order in which pairs are joined is fixed, so results do
// not depend on timing.  Where sequences begin, the state is replaced, and nothing behind it is
// looked at.

constexpr int CH = 4, LANES = SCAN_CHANNELS / CH;           // channels a lane; lanes of a row
constexpr int RUN = 8, RUNS = SCAN_ROWS / RUN;
static_assert(LANES * RUNS == 256, "a workgroup holds a segment");
constexpr uint32_t EMPTY = 0xffffffffu;                     // no log-decay has these bits
constexpr float CUT = 1.f;                                  // in place of a log-decay: a sequence began among the rows
constexpr int SPINS = 1 << 20;                              // about a second

struct Marks {
    int first[SCAN_ROWS], last[SCAN_ROWS];                  // the sequence that begins / ends at a row, or -1
    int any;
};

// Notes where sequences begin and end among rows [r0, r0 + SCAN_ROWS).  Sequences without rows that fall here (into
// the last segment: or behind it) get their resulting state at once, for channels [c0, c0 + SCAN_CHANNELS).
__device__ __forceinline__ void mark_rows(const ScanParams &p, int r0, bool tail, Marks &m, const float *from, float *to, int c0)
{
    const int t = threadIdx.x;
    if (t < SCAN_ROWS) m.first[t] = m.last[t] = -1;
    if (t == 0) m.any = 0;
    lds_barrier();
    const auto pass_on = [&](int s) {
        for (int c = c0; c < min(p.C, c0 + SCAN_CHANNELS); ++c) to[(size_t)s * p.C + c] = from ? from[(size_t)s * p.C + c] : 0.f;
    };
    bool any = false;
    if (!p.cu) {
        if (t < SCAN_ROWS && r0 + t < p.rows) {
            const int s = (r0 + t) / p.T, at = (r0 + t) - s * p.T;
            if (at == 0) m.first[t] = s;
            if (at == p.T - 1) m.last[t] = s;
            any = at == 0 || at == p.T - 1;
        }
        if (p.T == 0 && to)
            for (int s = t; s < p.N; s += 256) pass_on(s);
    } else {
        // of a long list, from the last sequence that begins before these rows
        int lo = 0;
        for (int hi = p.N; hi - lo > 1024;) {
            const int mid = (lo + hi) / 2;
            if (p.cu[mid] < r0) lo = mid; else hi = mid;
        }
        for (int s = lo + t; s < p.N; s += 256) {
            int a, b;
            sequence_of(p, s, &a, &b);
            if (a >= r0 + SCAN_ROWS && !tail) break;
            if (b > a) {
                if (a >= r0 && a < r0 + SCAN_ROWS) m.first[a - r0] = s, any = true;
                if (b > r0 && b <= r0 + SCAN_ROWS) m.last[b - 1 - r0] = s, any = true;
            } else if (to && a >= r0 && (a < r0 + SCAN_ROWS || tail)) {
                pass_on(s);
            }
        }
    }
    if (any) m.any = 1;
    lds_barrier();
}

// Bit i: row run * RUN + i has a mark.
__device__ __forceinline__ unsigned run_marks(const int *mark, int run)
{
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < RUN; ++i) bits |= (mark[run * RUN + i] >= 0 ? 1u : 0u) << i;
    return bits;
}

// Bit i: row r0 + run * RUN + i belongs to a sequence.
__device__ __forceinline__ unsigned run_rows(const ScanParams &p, int r)
{
    int lo = 0, hi = p.rows;
    if (p.cu) {
        lo = min(max(p.cu[0], 0), p.rows);
        hi = min(max(p.cu[p.N], 0), p.rows);
    }
    const int a = min(max(lo - r, 0), RUN), b = min(max(hi - r, 0), RUN);
    return (0xffu >> (8 - b)) & (0xffu << a) & 0xffu;
}

__device__ __forceinline__ uint64_t pair_of(float g, float h)
{
    const uint32_t gb = g != g ? 0x7fc00000u : __builtin_bit_cast(uint32_t, g);
    return (uint64_t)gb << 32 | __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ float pair_g(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)(v >> 32)); }
__device__ __forceinline__ float pair_h(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)v); }
__device__ __forceinline__ uint64_t peek(const uint64_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void publish(uint64_t *p, uint64_t v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");                          // before any wait that follows
}

// Waits for up to LOOK pairs at[0], at[-C], ...: n of them.  A wait that lasts about a second (another call writes to this
// call's workspace) is given up, by all waits of the call: the pair counts as a cut with NaN.
constexpr int LOOK = 8;
__device__ __forceinline__ void await_pairs(const ScanChain &k, const uint64_t *at, int C, int n, uint64_t *v)
{
    for (int spin = 0;; ++spin) {
        bool all = true;
#pragma unroll
        for (int u = 0; u < LOOK; ++u) v[u] = u < n ? peek(at - (size_t)u * C) : 0;
#pragma unroll
        for (int u = 0; u < LOOK; ++u) all = all && (uint32_t)(v[u] >> 32) != EMPTY;
        if (all) return;
        if ((spin & 63) == 63 &&
            (spin >= SPINS || __hip_atomic_load(k.gave_up, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))) {
            __hip_atomic_store(k.gave_up, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int u = 0; u < LOOK; ++u)
                if ((uint32_t)(v[u] >> 32) == EMPTY) v[u] = pair_of(CUT, __builtin_bit_cast(float, 0x7fc00000u));
            return;
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

// The state before segment q (in the order of the scan) in channel c.
__device__ __forceinline__ float state_before(const ScanChain &k, int q, int c, int C)
{
    const int base = q / k.group * k.group;                 // behind segment base - 1 the state is published whole
    float G = 0.f, h = 0.f;
    for (int j = q - 1; j >= base; j -= LOOK) {
        uint64_t v[LOOK];
        const int n = min(LOOK, j - base + 1);
        await_pairs(k, k.part + (size_t)j * C + c, C, n, v);
#pragma unroll
        for (int u = 0; u < LOOK; ++u) {
            if (u >= n) break;
            h = decay_apply(decay_code(G), pair_h(v[u]), h);
            if (pair_g(v[u]) > 0.f) return h;
            G += pair_g(v[u]);
        }
    }
    if (base == 0) return h;
    uint64_t v[LOOK];
    await_pairs(k, k.whole + (size_t)(base / k.group - 1) * C + c, C, 1, v);
    return decay_apply(decay_code(G), pair_h(v[0]), h);
}

struct Joined {
    float G[RUNS][SCAN_CHANNELS], h[RUNS][SCAN_CHANNELS];   // of each run, then of the runs before it
    float in[SCAN_CHANNELS];                                // the state before the segment
    unsigned ticket;
};

// Joins the runs of every channel in the order of the scan (BACK: the last run first) and gets the state before the
// segment.  need: that state is looked at (no sequence begins at the segment's first row).
template <bool CHAIN, bool BACK>
__device__ __forceinline__ void join_runs(const ScanParams &p, int q, int c0, bool need, Joined &s)
{
    lds_barrier();
    const int t = threadIdx.x, c = c0 + t;
    if (t < SCAN_CHANNELS) {
        float G = 0.f, h = 0.f;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int k = BACK ? RUNS - 1 - i : i;
            const float g1 = s.G[k][t], h1 = s.h[k][t];
            s.G[k][t] = G;
            s.h[k][t] = h;
            const bool cut = g1 > 0.f;
            h = cut ? h1 : decay_apply(decay_code(g1), h, h1);
            G = cut || G > 0.f ? CUT : G + g1;
        }
        if (CHAIN && c < p.C) {
            publish(p.chain.part + (size_t)q * p.C + c, pair_of(G, h));
            const bool hand_on = (q + 1) % p.chain.group == 0;
            float in = 0.f;
            if (q > 0 && (need || (hand_on && !(G > 0.f)))) in = state_before(p.chain, q, c, p.C);
            if (hand_on)
                publish(p.chain.whole + (size_t)(q / p.chain.group) * p.C + c,
                        pair_of(0.f, G > 0.f ? h : decay_apply(decay_code(G), in, h)));
            s.in[t] = in;
        }
    }
    lds_barrier();
}

// The state before run `run` in channels [4 l, 4 l + 4) of the segment.
template <bool CHAIN> __device__ __forceinline__ void state_of_run(const Joined &s, int run, int l, float *h)
{
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        h[i] = s.h[run][CH * l + i];
        if (CHAIN) {
            const float G = s.G[run][CH * l + i];
            if (!(G > 0.f)) h[i] = decay_apply(decay_code(G), s.in[CH * l + i], h[i]);
        }
    }
}

__device__ __forceinline__ void put_run(Joined &s, int run, int l, bool cut, const float *G, const float *h)
{
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        s.G[run][CH * l + i] = cut ? CUT : G[i];
        s.h[run][CH * l + i] = h[i];
    }
}

// The segment and channels of a workgroup; false: none left (never, unless another call writes to the workspace).
template <bool CHAIN> __device__ __forceinline__ bool take_segment(const ScanParams &p, Joined &s, int *q, int *c0)
{
    const unsigned wide = (p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS;
    unsigned at = blockIdx.x;
    if (CHAIN) {
        if (threadIdx.x == 0) s.ticket = __hip_atomic_fetch_add(p.chain.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        lds_barrier();
        at = __builtin_amdgcn_readfirstlane(s.ticket);
    }
    *q = (int)(at / wide);
    *c0 = (int)(at % wide) * SCAN_CHANNELS;
    return *q < p.chain.segments;
}

// Four channels as they are stored: elements, or codes with their scale.
template <typename T> struct Held {
    static constexpr int WORDS = sizeof(T);
    uint32_t v[WORDS];
    __device__ __forceinline__ void load(const Rows &m, size_t r, int C, int c, int n)
    {
        if (m.scales) {
            const int8_t *at = (const int8_t *)m.p + r * m.stride + c;
            if (n == CH) {
                typedef uint32_t u32_any __attribute__((aligned(1)));
                v[0] = *reinterpret_cast<const u32_any *>(at);
            } else {
                v[0] = 0;
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (i < n) v[0] |= (uint32_t)(uint8_t)at[i] << (8 * i);
            }
            v[1] = n > 0 ? __builtin_bit_cast(uint32_t, m.scales[r * act_groups(C) + c / ACT_GROUP]) : 0;
            return;
        }
        Raw4<T> raw;
        raw.load((const T *)m.p + r * m.stride + c, n);
        __builtin_memcpy(v, &raw, sizeof(raw));
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void get(bool packed, float *x) const
    {
        if (packed) {
            const float s = __builtin_bit_cast(float, v[1]);
#pragma unroll
            for (int i = 0; i < CH; ++i) x[i] = (float)(int8_t)(v[0] >> (8 * i)) * s;
            return;
        }
        Raw4<T> raw;
        __builtin_memcpy(&raw, v, sizeof(raw));
#pragma unroll
        for (int i = 0; i < CH; ++i) x[i] = raw[i];
    }
};

template <typename T, typename G, bool CHAIN, bool FULL>
__device__ __forceinline__ void scan_fwd_segment(const ScanParams &p, int q, int c0, Joined &s, Marks &m)
{
    const int l = threadIdx.x % LANES, run = threadIdx.x / LANES, c = c0 + l * CH;
    const int r0 = q * SCAN_ROWS, r1 = r0 + run * RUN;
    const int n = FULL ? CH : max(0, min(CH, p.C - c));
    Raw4<T> x[RUN];
    Raw4<G> z[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        const size_t r = r1 + i;
        const int k = FULL || r1 + i < p.rows ? n : 0;
        x[i].load((const T *)p.x.p + r * p.x.stride + c, k);
        z[i].load((const G *)p.g.p + r * p.g.stride + c, k);
    }
    float eA[CH];
    if (p.A_log) {
        load_f4(p.A_log + c, n, eA);
#pragma unroll
        for (int i = 0; i < CH; ++i) eA[i] = __expf(eA[i]);
    }
    mark_rows(p, r0, q == p.chain.segments - 1, m, p.h0, p.hT, c0);
    unsigned first = 0, last = 0;
    const unsigned rows = run_rows(p, r1);
    if (m.any) {
        first = run_marks(m.first, run);
        last = run_marks(m.last, run);
    }
    const bool need = m.first[0] < 0;
    const auto begin = [&](int i, float *h) {
        if (p.h0)
            load_f4(p.h0 + (size_t)m.first[run * RUN + i] * p.C + c, n, h);
        else
#pragma unroll
            for (int j = 0; j < CH; ++j) h[j] = 0.f;
    };
    float w[RUN][CH], g[CH] = {}, h[CH] = {};
    const bool gated = p.A_log != nullptr;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        if (first >> i & 1) begin(i, h);
        const bool in = rows >> i & 1;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float d = gated ? p.g_min * sigmoid2(eA[j] * z[i][j]).s : z[i][j];
            d = d > 0.f || !in ? 0.f : d;
            w[i][j] = decay_code(d);
            g[j] += d;
            const float b = !in ? 0.f : p.complement ? x[i][j] * decay_rest(w[i][j]) : x[i][j];
            h[j] = decay_apply(w[i][j], h[j], b);
        }
    }
    put_run(s, run, l, first != 0, g, h);
    join_runs<CHAIN, false>(p, q, c0, need, s);
    state_of_run<CHAIN>(s, run, l, h);
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        if (first >> i & 1) begin(i, h);
        const bool in = rows >> i & 1;
        float out[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const float b = !in ? 0.f : p.complement ? x[i][j] * decay_rest(w[i][j]) : x[i][j];
            h[j] = decay_apply(w[i][j], h[j], b);
            out[j] = h[j];
        }
        const size_t at = (size_t)(r1 + i) * p.C + c;
        if (in && n > 0) Raw4<T>::store((T *)p.h + at, n, out);
        if (p.h8.codes) {
#pragma unroll
            for (int j = 0; j < CH; ++j) out[j] = j < n ? to_f<T>(from_f<T>(out[j])) : 0.f;
            store_codes<CH>(p.h8, r1 + i, p.C, c, in ? n : 0, out);
        }
        if (last >> i & 1 && p.hT && n > 0) Raw4<float>::store(p.hT + (size_t)m.last[run * RUN + i] * p.C + c, n, h);
    }
}

template <typename T, typename G, bool CHAIN> __global__ __launch_bounds__(256, 4) void scan_fwd_kernel(const ScanParams p)
{
    __shared__ Joined s;
    __shared__ Marks m;
    int q, c0;
    if (!take_segment<CHAIN>(p, s, &q, &c0)) return;
    if (c0 + SCAN_CHANNELS <= p.C && (q + 1) * SCAN_ROWS <= p.rows)
        scan_fwd_segment<T, G, CHAIN, true>(p, q, c0, s, m);
    else
        scan_fwd_segment<T, G, CHAIN, false>(p, q, c0, s, m);
}

// Gradients, from the last row to the first: D_t = d_h_t + e_{t+1}, e_t = a_t D_t; runs, segments and their order mirrored.
template <typename T, typename G, bool CHAIN, bool FULL>
__device__ __forceinline__ void scan_bwd_segment(const ScanParams &p, int q, int c0, Joined &s, Marks &m)
{
    const int l = threadIdx.x % LANES, run = threadIdx.x / LANES, c = c0 + l * CH;
    const int r0 = (p.chain.segments - 1 - q) * SCAN_ROWS, r1 = r0 + run * RUN;
    const int n = FULL ? CH : max(0, min(CH, p.C - c));
    Raw4<T> d[RUN];
    Raw4<G> z[RUN];
    const auto there = [&](int i) { return FULL || r1 + i < p.rows ? n : 0; };
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        const size_t r = r1 + i;
        d[i].load((const T *)p.d_h + r * p.C + c, there(i));
        z[i].load((const G *)p.g.p + r * p.g.stride + c, there(i));
    }
    float eA[CH];
    if (p.A_log) {
        load_f4(p.A_log + c, n, eA);
#pragma unroll
        for (int i = 0; i < CH; ++i) eA[i] = __expf(eA[i]);
    }
    mark_rows(p, r0, q == 0, m, p.dhT, p.dh0, c0);
    unsigned first = 0, last = 0;
    const unsigned rows = run_rows(p, r1);
    if (m.any) {
        first = run_marks(m.first, run);
        last = run_marks(m.last, run);
    }
    const bool need = m.last[SCAN_ROWS - 1] < 0;
    const auto begin = [&](int i, float *e) {
        if (p.dhT)
            load_f4(p.dhT + (size_t)m.last[run * RUN + i] * p.C + c, n, e);
        else
#pragma unroll
            for (int j = 0; j < CH; ++j) e[j] = 0.f;
    };
    float w[RUN][CH], g[CH] = {}, e[CH] = {};
    const bool gated = p.A_log != nullptr;
#pragma unroll
    for (int i = RUN - 1; i >= 0; --i) {
        if (last >> i & 1) begin(i, e);
        const bool in = rows >> i & 1;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float x = gated ? p.g_min * sigmoid2(eA[j] * z[i][j]).s : z[i][j];
            x = x > 0.f || !in ? 0.f : x;
            w[i][j] = decay_code(x);
            g[j] += x;
            e[j] = decay_times(w[i][j], in ? d[i][j] + e[j] : e[j]);
        }
    }
    put_run(s, run, l, last != 0, g, e);
    Held<T> hs[RUN], xs[RUN];
    if (p.dg) {
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            // the row before; a sequence's first has none
            const size_t r = r1 + i;
            if (r > 0) hs[i].load(p.hs, r - 1, p.C, c, FULL || r1 + i - 1 < p.rows ? n : 0); else hs[i].clear();
            if (p.complement) xs[i].load(p.x, r, p.C, c, there(i));
        }
    }
    join_runs<CHAIN, true>(p, q, c0, need, s);
    state_of_run<CHAIN>(s, run, l, e);
    float dA[CH] = {};
#pragma unroll
    for (int i = RUN - 1; i >= 0; --i) {
        if (last >> i & 1) begin(i, e);
        const bool in = rows >> i & 1;
        float out[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const float D = in ? d[i][j] + e[j] : e[j];
            e[j] = decay_times(w[i][j], D);
            out[j] = p.complement ? D * decay_rest(w[i][j]) : D;
        }
        const size_t r = r1 + i;
        if (in && n > 0) Raw4<T>::store((T *)p.dx + r * p.dx_stride + c, n, out);
        if (p.dg) {
            float prev[CH];
            hs[i].get(p.hs.scales, prev);
            if (first >> i & 1) {
                if (p.h0)
                    load_f4(p.h0 + (size_t)m.first[run * RUN + i] * p.C + c, n, prev);
                else
#pragma unroll
                    for (int j = 0; j < CH; ++j) prev[j] = 0.f;
            }
            if (p.complement) {
                xs[i].get(p.x.scales, out);
#pragma unroll
                for (int j = 0; j < CH; ++j) prev[j] -= out[j];
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                out[j] = e[j] * prev[j];
                if (gated) {
                    const Sigmoid sg = sigmoid2(eA[j] * z[i][j]);
                    out[j] *= p.g_min * sg.s * sg.r * eA[j];
                    if (in) dA[j] += out[j] * z[i][j];
                }
            }
            if (in && n > 0) Raw4<G>::store((G *)p.dg + r * p.dg_stride + c, n, out);
        }
        if (first >> i & 1 && p.dh0 && n > 0) Raw4<float>::store(p.dh0 + (size_t)m.first[run * RUN + i] * p.C + c, n, e);
    }
    if (p.dA) {                                             // the segment's part of dA: runs in their order
        lds_barrier();
#pragma unroll
        for (int j = 0; j < CH; ++j) s.h[run][CH * l + j] = dA[j];
        lds_barrier();
        const int t = threadIdx.x;
        if (t < SCAN_CHANNELS && c0 + t < p.C) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < RUNS; ++k) sum += s.h[k][t];
            p.dA_part[(size_t)q * p.C + c0 + t] = sum;
        }
    }
}

template <typename T, typename G, bool CHAIN> __global__ __launch_bounds__(256, 2) void scan_bwd_kernel(const ScanParams p)
{
    __shared__ Joined s;
    __shared__ Marks m;
    int q, c0;
    if (!take_segment<CHAIN>(p, s, &q, &c0)) return;
    if (c0 + SCAN_CHANNELS <= p.C && (p.chain.segments - q) * SCAN_ROWS <= p.rows)
        scan_bwd_segment<T, G, CHAIN, true>(p, q, c0, s, m);
    else
        scan_bwd_segment<T, G, CHAIN, false>(p, q, c0, s, m);
}

// Clears the hand-over's memory (no pair there yet; ticket and flag, its last word, 0) and copies states that the call overwrites.
__global__ __launch_bounds__(256) void scan_clear_kernel(uint64_t *words, size_t n, const float *from, float *to, size_t states)
{
    const size_t step = (size_t)gridDim.x * 256;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) words[i] = i + 1 < n ? ~(uint64_t)0 : 0;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < states; i += step) to[i] = from[i];
}

// Sums of the segments' parts, in their order.
__global__ __launch_bounds__(256) void scan_sum_kernel(const float *part, int parts, int C, float *out)
{
    __shared__ double s_part[4][64];
    const int l = threadIdx.x & 63, c = blockIdx.x * 64 + l, slice = threadIdx.x / 64;
    double sum = 0.0;
    if (c < C)
        for (int i = slice; i < parts; i += 4) sum += part[(size_t)i * C + c];
    s_part[slice][l] = sum;
    __syncthreads();
    if (slice == 0 && c < C) out[c] = (float)((s_part[0][l] + s_part[1][l]) + (s_part[2][l] + s_part[3][l]));
}

// One token a sequence: 8 channels a lane.  Slots as for kda_linear_recurrent_step.
template <typename T, typename G> __global__ __launch_bounds__(256) void scan_step_kernel(const ScanStepParams p)
{
    const int blocks = (p.C + 2047) / 2048;
    const int n = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 2048 + threadIdx.x * LANE_CH;
    const int cnt = max(0, min(LANE_CH, p.C - c));
    int slot = n;
    bool mine = true;
    if (p.slots) {
        slot = p.slots[n];
        mine = slot >= 0 && slot < p.n_slots;
        bool seen = false;
        for (int j = threadIdx.x; j < n; j += 256) seen |= p.slots[j] == slot;
        mine = !__syncthreads_or(seen) && mine;
    }
    if (cnt == 0) return;
    float h[8];
    if (mine) {
        Raw8<T> x;
        Raw8<G> g;
        float A[8];
        x.load((const T *)p.x.p + n * p.x.stride + c, cnt);
        g.load((const G *)p.g.p + n * p.g.stride + c, cnt);
        load_f8(p.state + (size_t)slot * p.C + c, cnt, h);
        if (p.A_log) load_f8(p.A_log + c, cnt, A);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = decay_code(p.A_log ? p.g_min * sigmoid2(__expf(A[i]) * g[i]).s : g[i]);
            h[i] = decay_apply(w, h[i], p.complement ? x[i] * decay_rest(w) : x[i]);
        }
        Raw8<float>::store(p.new_state + (size_t)slot * p.C + c, cnt, h);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = 0.f;
    }
    Raw8<T>::store((T *)p.h + (size_t)n * p.C + c, cnt, h);
}

static hipError_t launch_clear(const ScanParams &p, const float *states, hipStream_t stream)
{
    const size_t copied = p.state_copy ? (size_t)p.N * p.C : 0;
    const size_t most = p.chain.words > copied ? p.chain.words : copied;
    if (most == 0) return hipSuccess;
    const size_t grid = (most + 1023) / 1024;
    hipLaunchKernelGGL(scan_clear_kernel, dim3((unsigned)(grid < 1024 ? grid : 1024)), dim3(256), 0, stream, p.chain.part, p.chain.words, states,
                       p.state_copy, copied);
    return hipGetLastError();
}

template <typename T, typename G> static hipError_t launch_fwd_t(ScanParams p, hipStream_t stream)
{
    const dim3 grid((unsigned)p.chain.segments * ((p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS));
    const hipError_t e = launch_clear(p, p.h0, stream);
    if (e != hipSuccess) return e;
    if (p.state_copy) p.h0 = p.state_copy;
    if (p.chain.words)
        hipLaunchKernelGGL((scan_fwd_kernel<T, G, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((scan_fwd_kernel<T, G, false>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <typename T, typename G> static hipError_t launch_bwd_t(ScanParams p, hipStream_t stream)
{
    const dim3 grid((unsigned)p.chain.segments * ((p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS));
    const hipError_t e = launch_clear(p, p.dhT, stream);
    if (e != hipSuccess) return e;
    if (p.state_copy) p.dhT = p.state_copy;
    if (p.chain.words)
        hipLaunchKernelGGL((scan_bwd_kernel<T, G, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((scan_bwd_kernel<T, G, false>), grid, dim3(256), 0, stream, p);
    if (p.dA)
        hipLaunchKernelGGL(scan_sum_kernel, dim3((p.C + 63) / 64), dim3(256), 0, stream, p.dA_part, p.chain.segments, p.C, p.dA);
    return hipGetLastError();
}

template <typename T, typename G> static hipError_t launch_step_t(const ScanStepParams &p, hipStream_t stream)
{
    hipLaunchKernelGGL((scan_step_kernel<T, G>), dim3((unsigned)p.N * ((p.C + 2047) / 2048)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

#define KDA_SCAN_CASE(fn)                                                                       \
    return !is_bf16 ? fn<float, float>(p, stream) : g_bf16 ? fn<bf16, bf16>(p, stream) : fn<bf16, float>(p, stream)

hipError_t launch_scan_fwd(int is_bf16, int g_bf16, const ScanParams &p, hipStream_t stream) { KDA_SCAN_CASE(launch_fwd_t); }
hipError_t launch_scan_bwd(int is_bf16, int g_bf16, const ScanParams &p, hipStream_t stream) { KDA_SCAN_CASE(launch_bwd_t); }
hipError_t launch_scan_step(int is_bf16, int g_bf16, const ScanStepParams &p, hipStream_t stream) { KDA_SCAN_CASE(launch_step_t); }

#undef KDA_SCAN_CASE

}  // namespace kda

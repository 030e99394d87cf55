// kda_scan.hip -- the gated scan  h_t = a_t h_{t-1} + m_t x_t  per channel:
// whole sequences, their gradients, one token.
#include <float.h>

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
// h_t = a_t h_{t-1} + b_t is associative: a run of tokens maps the state before it to (product of a) h + (state from
// zero).  A workgroup takes 64 rows of 128 channels: 32 lanes hold 4 channels each, 8 groups of lanes 8 rows each.  A
// lane runs over its rows from zero (keeping the decays), 128 threads join the 8 runs of a channel through LDS, and with
// the state before it each lane runs over its rows again from registers: x and g are read once, h written once.  That
// takes 128 registers forwards and 151 backwards in bf16: four and three waves a SIMD.
//
// Segments of a call's packed rows are joined in the same pass.  Workgroups take tickets of their channels (so a
// segment's predecessors run or have run already) and publish what their rows do to a state, a pair (product of decays,
// state from zero), before waiting for anything.  The last segment of every 8 joins these pairs and publishes the
// block's; the last of every 64 publishes the state behind it.  So a segment waits for at most 7 pairs of its block, 7 of
// blocks and one state, and what has to pass from one to the next is one state every 4096 rows (one in every 512: 6%
// slower).  The order in which pairs are joined is fixed, so results do not depend on timing.  Where sequences begin, the
// state is replaced, and what lies before is not waited for.
//
// Bound by no unit alone: a workgroup's load, pass, wait and store follow one another, and the four of a compute unit do not fill each
// other's gaps.  131072 rows x 2048 in bf16 with the gate take 504 us (3.2 TB/s; a copy would take 327), of which the vector units issue
// 61% of the time and a wave waits 61% (38 instructions a token with the gate, all passes and the hand-over).  8192 x 4096: 62 us, 70 on
// tensors that no cache holds, without the gate 66; gradients 104 us, from 8-bit values 98 (vector units 77%).  With an odd number of channels
// vectors are read at odd addresses: 8192 x 4001 77 and 154 us.
// One segment has nothing to join: no tickets, no clearing (one launch less, 13.4 us instead of 17 with the call).

constexpr int CH = 4, LANES = SCAN_CHANNELS / CH;           // channels a lane; lanes of a row
constexpr int RUN = 8, RUNS = SCAN_ROWS / RUN;
static_assert(LANES * RUNS == 256, "a workgroup holds a segment");
constexpr uint32_t EMPTY = 0xffffffffu;                     // no decay has these bits
constexpr float CUT = 2.f;                                  // in place of a decay: a sequence began among the rows
constexpr int BLOCK = SCAN_BLOCK;
constexpr int TICKET_STEP = SCAN_TICKET_STEP;
constexpr int SPINS = 1 << 20;                              // some tenths of a second

struct Marks {
    int first[SCAN_ROWS], last[SCAN_ROWS];                  // the sequence that begins / ends at a row, or -1
    int any;
};

// What a thread needs of the offsets, loaded ahead of the segment's values: memory answers in order.
struct Offsets {
    int lo, a, b, begin, end;                               // rows [a, b) of sequence lo + thread; of all sequences
    __device__ __forceinline__ Offsets(const ScanParams &p, int r0)
    {
        lo = a = b = begin = 0;
        end = p.rows;
        if (!p.cu) return;
        // of a long list, from the last sequence that begins before these rows
        for (int hi = p.N; hi - lo > 1024;) {
            const int mid = (lo + hi) / 2;
            if (p.cu[mid] < r0) lo = mid; else hi = mid;
        }
        if (lo + (int)threadIdx.x < p.N) sequence_of(p, lo + threadIdx.x, &a, &b);
        begin = min(max(p.cu[0], 0), p.rows);
        end = min(max(p.cu[p.N], 0), p.rows);
    }
};

// Notes where sequences begin and end among rows [r0, r0 + SCAN_ROWS).  Of up to SCAN_MANY sequences those without rows that fall here (into
// the last segment: or behind it) get their resulting state at once, for channels [c0, c0 + SCAN_CHANNELS).
__device__ __forceinline__ void mark_rows(const ScanParams &p, const Offsets &o, int r0, bool tail, Marks &m, const float *from,
                                          float *to, int c0)
{
    const int t = threadIdx.x;
    if (t < SCAN_ROWS) m.first[t] = m.last[t] = -1;
    if (t == 0) m.any = 0;
    lds_barrier();
    if (!p.cu && p.T > 0 && r0 % p.T != 0 && r0 % p.T + SCAN_ROWS < p.T) return;   // inside a sequence
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
    } else if (p.N > SCAN_MANY) {
        const int r = r0 + t;
        if (t < SCAN_ROWS && r < p.rows) {
            int s = o.lo, a, b;                             // the last sequence that begins at row r or before
            for (int hi = p.N; hi - s > 1;) {
                const int mid = s + (hi - s) / 2;
                if (p.cu[mid] <= r) s = mid; else hi = mid;
            }
            sequence_of(p, s, &a, &b);
            if (r == a && b > a) m.first[t] = s, any = true;
            if (r == b - 1 && b > a) m.last[t] = s, any = true;
        }
    } else {
        int a = o.a, b = o.b;
        for (int s = o.lo + t; s < p.N; s += 256) {
            if (s != o.lo + t) sequence_of(p, s, &a, &b);
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

// Bit i: row r + i belongs to a sequence.
__device__ __forceinline__ unsigned run_rows(const Offsets &o, int r)
{
    const int a = min(max(o.begin - r, 0), RUN), b = min(max(o.end - r, 0), RUN);
    return (0xffu >> (8 - b)) & (0xffu << a) & 0xffu;
}

__device__ __forceinline__ uint64_t pair_of(float w, float h)
{
    const uint32_t wb = w != w ? 0x7fc00000u : __builtin_bit_cast(uint32_t, w);
    return (uint64_t)wb << 32 | __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ float pair_w(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)(v >> 32)); }
__device__ __forceinline__ float pair_h(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)v); }
__device__ __forceinline__ float join(float w, float h1, float h) { return w == CUT ? h1 : decay_apply(decay_held(w), h, h1); }
__device__ __forceinline__ uint64_t peek(const uint64_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void publish(uint64_t *p, uint64_t v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");                          // before any wait that follows
}

// Waits for the pairs at(0) .. at(n - 1), n <= BLOCK.  A wait that lasts some tenths of a second (another call writes to this call's
// workspace) is given up, by all waits of the call: the pair counts as a cut with NaN.
template <typename F> __device__ __forceinline__ void await_pairs(const ScanChain &k, int n, F at, uint64_t *v)
{
    for (int spin = 0;; ++spin) {
        bool all = true;
#pragma unroll
        for (int u = 0; u < BLOCK; ++u)
            if (u < n) v[u] = peek(at(u));
#pragma unroll
        for (int u = 0; u < BLOCK; ++u) all = all && (u >= n || (uint32_t)(v[u] >> 32) != EMPTY);
        if (all) return;
        if ((spin & 63) == 63 &&
            (spin >= SPINS || __hip_atomic_load(k.gave_up, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))) {
            __hip_atomic_store(k.gave_up, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int u = 0; u < BLOCK; ++u)
                if (u < n && (uint32_t)(v[u] >> 32) == EMPTY) v[u] = pair_of(CUT, __builtin_bit_cast(float, 0x7fc00000u));
            return;
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

struct Joined {
    float w[RUNS][SCAN_CHANNELS], h[RUNS][SCAN_CHANNELS];   // of each run; then the state before it from the segment's
    float G[RUNS][SCAN_CHANNELS];                           // log-decay of a run, then of the runs before it (cut: +1)
    float in[SCAN_CHANNELS];                                // the state before the segment's block, then before the segment
    unsigned ticket;
};

// Joins the runs of every channel in the order of the scan (BACK: the last run first) and gets the state before the
// segment.  need: that state is looked at (no sequence begins at the segment's first row).  Waves 0 and 1 join, publish and wait for the
// segments of the block, the other two for what lies before the block.
template <bool CHAIN, bool BACK>
__device__ __forceinline__ void join_runs(const ScanParams &p, int q, int c0, bool need, Joined &s)
{
    lds_barrier();
    const ScanChain &k = p.chain;
    const int block = q / BLOCK, n = q % BLOCK;             // of the segments; n of the block lie before
    const bool ends_block = n == BLOCK - 1, ends_all = ends_block && block % BLOCK == BLOCK - 1;
    const bool joins = threadIdx.x < SCAN_CHANNELS;
    const unsigned t = joins ? threadIdx.x : threadIdx.x - SCAN_CHANNELS, c = c0 + t;
    const bool there = CHAIN && c < (unsigned)p.C;
    need = need && q > 0;
    float w = 0.f, h = 0.f;
    uint64_t v[BLOCK];
    if (joins) {
        float G = 0.f;
        bool cut = false;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int j = BACK ? RUNS - 1 - i : i;
            const float g1 = s.G[j][t], w1 = s.w[j][t], h1 = s.h[j][t];
            s.G[j][t] = cut ? 1.f : G;
            s.h[j][t] = h;
            h = join(w1, h1, h);
            cut = cut || w1 == CUT;
            G += g1;
        }
        w = cut ? CUT : decay_of(not_above_0(G)).w;
        if (there) {
            publish(k.part + (size_t)q * p.C + c, pair_of(w, h));
            if (n > 0 && (need || ends_block))
                await_pairs(k, n, [&](int u) { return k.part + (size_t)(q - n + u) * p.C + c; }, v);
            if (ends_block) {
                float to = pair_h(v[0]);
                Decay all = decay_held(pair_w(v[0]));
                cut = pair_w(v[0]) == CUT;
#pragma unroll
                for (int u = 1; u < BLOCK - 1; ++u) {
                    cut = cut || pair_w(v[u]) == CUT;
                    to = join(pair_w(v[u]), pair_h(v[u]), to);
                    all = decay_product(all, decay_held(pair_w(v[u])));
                }
                const float bw = w == CUT || cut ? CUT : decay_product(all, decay_held(w)).w;
                publish(k.blocks + (size_t)block * p.C + c, pair_of(bw, join(w, h, to)));
            }
        }
    } else if (there) {
        float in = 0.f;
        if ((need || ends_all) && block > 0) {
            const int b0 = block / BLOCK * BLOCK, before = b0 > 0;
            await_pairs(k, before + block - b0, [&](int u) {
                return u < before ? k.whole + (size_t)(b0 / BLOCK - 1) * p.C + c : k.blocks + (size_t)(b0 + u - before) * p.C + c;
            }, v);
            // the state behind the blocks before counts as a cut: pair (2, state)
#pragma unroll
            for (int u = 0; u < BLOCK; ++u)
                if (u < before + block - b0) in = join(pair_w(v[u]), pair_h(v[u]), in);
        }
        s.in[t] = in;
    }
    lds_barrier();
    if (CHAIN) {
        if (joins && there) {
            float in = s.in[t];
            if (need)
#pragma unroll
                for (int u = 0; u < BLOCK - 1; ++u)
                    if (u < n) in = join(pair_w(v[u]), pair_h(v[u]), in);
            if (ends_all) {
                // (without need the segment is a cut)
                publish(k.whole + (size_t)(block / BLOCK) * p.C + c, pair_of(CUT, join(w, h, in)));
            }
            s.in[t] = in;
        }
        lds_barrier();
    }
}

// The state before run `run` in channels [4 l, 4 l + 4) of the segment.
template <bool CHAIN> __device__ __forceinline__ void state_of_run(const Joined &s, int run, int l, float *h)
{
#pragma unroll
    for (int i = 0; i < CH; ++i) h[i] = s.h[run][CH * l + i];
    if (CHAIN && !(s.G[run][CH * l] > 0.f)) {               // cuts are rows': the same in all channels
#pragma unroll
        for (int i = 0; i < CH; ++i) h[i] = decay_apply(decay_of(not_above_0(s.G[run][CH * l + i])), s.in[CH * l + i], h[i]);
    }
}

__device__ __forceinline__ void put_run(Joined &s, int run, int l, bool cut, const float *G, const float *h)
{
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        s.G[run][CH * l + i] = G[i];
        s.w[run][CH * l + i] = cut ? CUT : decay_of(not_above_0(G[i])).w;
        s.h[run][CH * l + i] = h[i];
    }
}

// A lane's part of a segment in memory: rows of CH channels, at 32-bit offsets from the segment's first element
// (64 rows of at most 2^24 elements).  In segments whose channels all exist, or whose C is a multiple of CH, every lane reads whole
// vectors (a lane or row without elements those of the last that has some, and nothing looks at them); in others every lane
// goes element by element, the last one again in place of those that are not there
// (with a condition for each element instead, whose loads wait for one another, 8192 x 4001 took 86 us and its gradients 171).
struct Window {
    int rows, n;                                            // rows of the segment that there are; the lane's channels
    bool vec, full;                                         // full: all channels of the segment exist
    int row0;                                               // the lane's first row
    unsigned col;
    __device__ __forceinline__ Window(const ScanParams &p, int r0, int c0)
    {
        const int c = c0 + (threadIdx.x % LANES) * CH;
        rows = min(p.rows - r0, SCAN_ROWS);
        n = max(0, min(CH, p.C - c));
        full = c0 + SCAN_CHANNELS <= p.C;
        vec = full || p.C % CH == 0;
        row0 = (threadIdx.x / LANES) * RUN;
        col = (vec ? min(c, p.C - CH) : min(c, p.C - 1)) - c0;
    }
    template <typename T> __device__ __forceinline__ void load(Raw4<T> *raw, const T *base, int64_t stride) const
    {
        const unsigned end = (unsigned)(rows - 1) * (unsigned)stride;
        unsigned off = (unsigned)row0 * (unsigned)stride;
        const auto rows_of = [&](auto load_row) {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                load_row(raw[i], base + (min(off, end) + col));
                off += (unsigned)stride;
                asm("" : "+v"(off));                        // one addition a row, not a product
            }
        };
        if (vec)
            rows_of([&](Raw4<T> &r, const T *p) { r.load(p, CH); });
        else
            rows_of([&](Raw4<T> &r, const T *p) {
#pragma unroll
                for (int j = 0; j < CH; ++j) r.v[j] = p[element(j)];
            });
    }
    // Of the lane's channels, where they are not read as a vector.
    __device__ __forceinline__ unsigned element(int j) const { return min(j, max(n, 1) - 1); }
    template <typename T> __device__ __forceinline__ void put(T *at, const float *x) const
    {
        if (vec) {
            if (n > 0) Raw4<T>::store(at, CH, x);
        } else {
            if (n > 0) Raw4<T>::store(at, n, x);
        }
    }
};

// The lane's rows of an array one after the other, up or down.
template <typename T> struct Cursor {
    T *base;
    unsigned off, step;
    __device__ __forceinline__ Cursor(T *b, const Window &w, int64_t stride, int i)
        : base(b), off((unsigned)(w.row0 + i) * (unsigned)stride + w.col), step((unsigned)stride) {}
    __device__ __forceinline__ T *at() const { return reinterpret_cast<T *>(reinterpret_cast<char *>(base) + off * (unsigned)sizeof(T)); }
    __device__ __forceinline__ void up() { off += step; asm("" : "+v"(off)); }
    __device__ __forceinline__ void down() { off -= step; asm("" : "+v"(off)); }
};

// Four channels as they are stored: elements, or codes with their scale.
template <typename T> struct Held {
    static constexpr int WORDS = sizeof(T);
    uint32_t v[WORDS];
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

// How a backward call's saved activations are stored: known to the kernel they take half the registers of either case.
enum Saved { ELEMENTS, CODES, EITHER };
template <Saved S> __device__ __forceinline__ bool is_packed(const Rows &m) { return S == CODES || (S == EITHER && m.scales); }

// The lane's rows of the segment from row r0 on, or (BEFORE) the rows before them, where there is one.
template <bool BEFORE, Saved S, typename T>
__device__ __forceinline__ void load_held(Held<T> *to, const Window &w, const Rows &m, int r0, int c0, int C)
{
    const int base = BEFORE && r0 > 0 ? r0 - 1 : r0, skip = BEFORE && r0 == 0;
    const unsigned stride = (unsigned)m.stride;
    if (is_packed<S>(m)) {
        const int8_t *codes = (const int8_t *)m.p + (size_t)base * m.stride + c0;
        const float *scales = m.scales + (size_t)base * act_groups(C) + c0 / ACT_GROUP;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const unsigned r = (unsigned)max(min(w.row0 + i, w.rows - 1) - skip, 0);
            const int8_t *at = codes + (r * stride + w.col);
            to[i].v[0] = 0;
            if (w.vec) {
                typedef uint32_t u32_any __attribute__((aligned(1)));
                to[i].v[0] = *reinterpret_cast<const u32_any *>(at);
            } else {
#pragma unroll
                for (int j = 0; j < CH; ++j) to[i].v[0] |= (uint32_t)(uint8_t)at[w.element(j)] << (8 * j);
            }
            to[i].v[1] = __builtin_bit_cast(uint32_t, scales[r * (unsigned)act_groups(C)]);
        }
        return;
    }
    const T *rows = (const T *)m.p + (size_t)base * m.stride + c0;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        const unsigned r = (unsigned)max(min(w.row0 + i, w.rows - 1) - skip, 0);
        Raw4<T> raw;
        const T *at = rows + (r * stride + w.col);
        if (w.vec)
            raw.load(at, CH);
        else
#pragma unroll
            for (int j = 0; j < CH; ++j) raw.v[j] = at[w.element(j)];
        __builtin_memcpy(to[i].v, &raw, sizeof(raw));
    }
}

// A channel's gate (eq. (5)), or log-decays as they are.  The decay is made from u = Sigmoid(exp(A) z), of which the
// log-decay is g_min times, or from the log-decay itself.
template <bool GATED> struct Gates {
    float k[CH];                                            // -e^A log2(e)
    float c0, c1, c2, c3, border, to_log2;                  // decay_of's, for u (uniform)
    __device__ __forceinline__ void load(const Window &win, const float *A_log, int c0_)
    {
        if (!GATED) return;
        Raw4<float> raw;
        if (win.vec)
            raw.load(A_log + c0_ + win.col, CH);
        else
#pragma unroll
            for (int j = 0; j < CH; ++j) raw.v[j] = A_log[c0_ + win.col + win.element(j)];
#pragma unroll
        for (int j = 0; j < CH; ++j) k[j] = raw[j];
    }
    __device__ __forceinline__ void make(float g_min)
    {
        if (!GATED) return;
#pragma unroll
        for (int j = 0; j < CH; ++j) k[j] = __expf(k[j]) * -LOG2E;
        c0 = g_min;
        c1 = NEAR1 * g_min * g_min;
        c2 = NEAR2 * g_min * g_min * g_min;
        c3 = NEAR3 * (g_min * g_min) * (g_min * g_min);
        border = NEAR / g_min;
        to_log2 = g_min * LOG2E;
    }
    __device__ __forceinline__ float open(float z, int j) const
    {
        return GATED ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * k[j])) : not_above_0(z);
    }
    __device__ __forceinline__ Decay decay(float u) const
    {
        if (!GATED) return decay_of(u);
        const float m = u * __builtin_fmaf(u, __builtin_fmaf(u, __builtin_fmaf(u, c3, c2), c1), c0);
        const bool near = u < border;
        return {near ? m : __builtin_amdgcn_exp2f(u * to_log2), near};
    }
    // d log_decay / d z, but for g_min e^A
    __device__ __forceinline__ float slope(float z, int j) const
    {
        // e^-|y| (1 / (1 + e^-|y|))^2: 0 far out on either side
        const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(z * k[j])), s = __builtin_amdgcn_rcpf(1.f + e);
        return s * (e * s);
    }
};

struct Yes { static constexpr bool on = true; };
struct No { static constexpr bool on = false; };

// What is made from these words is not kept.
template <typename R> __device__ __forceinline__ void hold(R &raw)
{
    static_assert(sizeof(R) % 4 == 0, "whole registers");
#pragma unroll
    for (int i = 0; i < (int)(sizeof(R) / 4); ++i) asm volatile("" : "+v"(reinterpret_cast<uint32_t *>(&raw)[i]));
}

// The segment a workgroup takes of its column of channels, by a ticket of that column; false: none (never, unless another call
// writes to this call's workspace).
template <bool CHAIN> __device__ __forceinline__ bool take_segment(const ScanParams &p, int column, Joined &s, int *q)
{
    *q = 0;
    if (CHAIN) {
        if (threadIdx.x == 0)
            s.ticket = __hip_atomic_fetch_add(p.chain.tickets + (size_t)column * TICKET_STEP, 1u, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
        lds_barrier();
        *q = (int)__builtin_amdgcn_readfirstlane(s.ticket);
    }
    return (unsigned)*q < (unsigned)p.chain.segments;
}

// Forward.  Each pass has a form for segments that lie inside a sequence and whose channels all exist, with no questions asked,
// and one for all others.
template <typename T, typename G, bool GATED, bool CHAIN>
__global__ __launch_bounds__(256, sizeof(T) + sizeof(G) == 4 ? 4 : 3) void scan_fwd_kernel(const ScanParams p)
{
    __shared__ Joined s;
    __shared__ Marks m;
    const int column = blockIdx.x % ((p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS), c0 = column * SCAN_CHANNELS;
    int q;
    if (!take_segment<CHAIN>(p, column, s, &q)) return;
    const int l = threadIdx.x % LANES, run = threadIdx.x / LANES, r0 = q * SCAN_ROWS, c = c0 + l * CH;
    const Window win(p, r0, c0);
    const bool complement = p.complement;
    const Offsets offsets(p, r0);
    Gates<GATED> gates;
    gates.load(win, p.A_log, c0);
    Raw4<T> x[RUN];
    Raw4<G> z[RUN];
    if (p.rows > 0) {
        win.load<T>(x, (const T *)p.x.p + (size_t)r0 * p.x.stride + c0, p.x.stride);
        win.load<G>(z, (const G *)p.g.p + (size_t)r0 * p.g.stride + c0, p.g.stride);
    }
    mark_rows(p, offsets, r0, q == p.chain.segments - 1, m, p.h0, p.hT, c0);
    gates.make(p.g_min);
    const bool plain = m.any == 0 && r0 >= offsets.begin && r0 + SCAN_ROWS <= offsets.end && win.full;
    unsigned first = 0, last = 0, rows = 0;
    if (!plain) {
        rows = run_rows(offsets, r0 + win.row0);
        first = run_marks(m.first, run);
        last = run_marks(m.last, run);
    }
    const auto begin = [&](int i, float *h) {
        if (p.h0)
            load_f4(p.h0 + (size_t)m.first[run * RUN + i] * p.C + c, win.n, h);
        else
#pragma unroll
            for (int j = 0; j < CH; ++j) h[j] = 0.f;
    };
    float w[RUN][CH], v[RUN][CH], h[CH] = {};
    const auto pass = [&](auto free) {
        float g[CH] = {};
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            if (!free.on) {
                if (first >> i & 1) begin(i, h);
                if (!(rows >> i & 1)) continue;
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const float u = gates.open(z[i][j], j);
                const Decay d = gates.decay(u);
                w[i][j] = d.w;
                g[j] += u;
                v[i][j] = x[i][j];
                h[j] = decay_step(d, h[j], v[i][j], complement);
            }
        }
        if (GATED)
#pragma unroll
            for (int j = 0; j < CH; ++j) g[j] *= p.g_min;
        put_run(s, run, l, !free.on && first != 0, g, h);
    };
    if (plain) pass(Yes{}); else pass(No{});
    join_runs<CHAIN, false>(p, q, c0, m.first[0] < 0, s);
    state_of_run<CHAIN>(s, run, l, h);
    const auto finish = [&](auto free) {
        Cursor<T> out((T *)p.h + (size_t)r0 * p.C + c0, win, p.C, 0);
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const bool in = free.on || (rows >> i & 1);
            if (!free.on && (first >> i & 1)) begin(i, h);
            if (in) {
#pragma unroll
                for (int j = 0; j < CH; ++j) h[j] = decay_step(decay_held(w[i][j]), h[j], v[i][j], complement);
                if (free.on) Raw4<T>::store(out.at(), CH, h); else win.put(out.at(), h);
            }
            out.up();
            if (p.h8.codes) {
                float o[CH];
#pragma unroll
                for (int j = 0; j < CH; ++j) o[j] = free.on || j < win.n ? to_f<T>(from_f<T>(h[j])) : 0.f;
                store_codes<CH>(p.h8, r0 + win.row0 + i, p.C, c, free.on ? CH : in ? win.n : 0, o);
            }
            if (!free.on && (last >> i & 1) && p.hT && win.n > 0)
                Raw4<float>::store(p.hT + (size_t)m.last[run * RUN + i] * p.C + c, win.n, h);
        }
    };
    if (plain) finish(Yes{}); else finish(No{});
}

// Gradients, from the last row to the first: D_t = d_h_t + e_{t+1}, e_t = a_t D_t; runs, segments and their order mirrored.
// h and x are asked for before the wait.  Saved values of a kind that the kernel knows leave room for three waves a SIMD: 8192 x 4096
// 104 us in bf16, 98 from 8 bits; with a kernel for either, at the time, 180 instead of 114 and 132 instead of 110.  One
// that finds h in one form and x in the other, or a single segment, takes that kernel.
template <typename T, typename G, bool GATED, bool CHAIN, Saved S>
__global__ __launch_bounds__(256, sizeof(T) + sizeof(G) == 4 && S != EITHER ? 3 : 2) void scan_bwd_kernel(const ScanParams p)
{
    __shared__ Joined s;
    __shared__ Marks m;
    const int column = blockIdx.x % ((p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS), c0 = column * SCAN_CHANNELS;
    int q;
    if (!take_segment<CHAIN>(p, column, s, &q)) return;
    __builtin_amdgcn_s_setprio(2);                          // others wait for what comes before the join (99 us for 102)
    const int l = threadIdx.x % LANES, run = threadIdx.x / LANES, r0 = (p.chain.segments - 1 - q) * SCAN_ROWS, c = c0 + l * CH;
    const Window win(p, r0, c0);
    const bool complement = p.complement;
    const Offsets offsets(p, r0);
    Gates<GATED> gates;
    gates.load(win, p.A_log, c0);
    Raw4<T> d[RUN];
    Raw4<G> z[RUN];
    if (p.rows > 0) {
        win.load<T>(d, (const T *)p.d_h + (size_t)r0 * p.C + c0, p.C);
        win.load<G>(z, (const G *)p.g.p + (size_t)r0 * p.g.stride + c0, p.g.stride);
    }
    mark_rows(p, offsets, r0, q == 0, m, p.dhT, p.dh0, c0);
    gates.make(p.g_min);
    const bool plain = m.any == 0 && r0 >= offsets.begin && r0 + SCAN_ROWS <= offsets.end && win.full;
    unsigned first = 0, last = 0, rows = 0;
    if (!plain) {
        rows = run_rows(offsets, r0 + win.row0);
        first = run_marks(m.first, run);
        last = run_marks(m.last, run);
    }
    const auto begin = [&](int i, float *e) {
        if (p.dhT)
            load_f4(p.dhT + (size_t)m.last[run * RUN + i] * p.C + c, win.n, e);
        else
#pragma unroll
            for (int j = 0; j < CH; ++j) e[j] = 0.f;
    };
    float w[RUN][CH], e[CH] = {};
    const auto pass = [&](auto free) {
        float g[CH] = {};
#pragma unroll
        for (int i = RUN - 1; i >= 0; --i) {
            if (!free.on) {
                if (last >> i & 1) begin(i, e);
                if (!(rows >> i & 1)) continue;
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const float u = gates.open(z[i][j], j);
                const Decay k = gates.decay(u);
                w[i][j] = k.w;
                g[j] += u;
                e[j] = decay_times(k, d[i][j] + e[j]);
            }
        }
        if (GATED)
#pragma unroll
            for (int j = 0; j < CH; ++j) g[j] *= p.g_min;
        put_run(s, run, l, !free.on && last != 0, g, e);
    };
    if (plain) pass(Yes{}); else pass(No{});
    // the second pass unpacks them again: 16 bits a value instead of 32 while the segment waits
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        hold(d[i]);
        hold(z[i]);
    }
    Held<T> hs[RUN], xs[RUN];
    if (p.dg && p.rows > 0) {
        load_held<true, S>(hs, win, p.hs, r0, c0, p.C);
        if (p.complement) load_held<false, S>(xs, win, p.x, r0, c0, p.C);
    }
    join_runs<CHAIN, true>(p, q, c0, m.last[SCAN_ROWS - 1] < 0, s);
    state_of_run<CHAIN>(s, run, l, e);
    float dA[CH] = {}, unit[CH];
    if (GATED)
#pragma unroll
        for (int j = 0; j < CH; ++j) unit[j] = p.g_min * gates.k[j] * (-1.f / LOG2E);
    const auto finish = [&](auto free) {
        Cursor<T> to_x((T *)p.dx + (size_t)r0 * p.dx_stride + c0, win, p.dx_stride, RUN - 1);
        Cursor<G> to_g((G *)p.dg + (size_t)r0 * p.dg_stride + c0, win, p.dg_stride, RUN - 1);
#pragma unroll
        for (int i = RUN - 1; i >= 0; --i) {
            if (!free.on && (last >> i & 1)) begin(i, e);
            if (free.on || (rows >> i & 1)) {
                float out[CH];
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    const Decay k = decay_held(w[i][j]);
                    const float D = d[i][j] + e[j];
                    e[j] = decay_times(k, D);
                    out[j] = share_of(k, D, complement);
                }
                if (free.on) Raw4<T>::store(to_x.at(), CH, out); else win.put(to_x.at(), out);
                if (p.dg) {
                    float prev[CH];
                    hs[i].get(is_packed<S>(p.hs), prev);
                    if (!free.on && (first >> i & 1)) {
                        if (p.h0)
                            load_f4(p.h0 + (size_t)m.first[run * RUN + i] * p.C + c, win.n, prev);
                        else
#pragma unroll
                            for (int j = 0; j < CH; ++j) prev[j] = 0.f;
                    }
                    if (p.complement) {
                        xs[i].get(is_packed<S>(p.x), out);
#pragma unroll
                        for (int j = 0; j < CH; ++j) prev[j] -= out[j];
                    }
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        out[j] = e[j] * prev[j];
                        if (GATED) {
                            out[j] *= unit[j] * gates.slope(z[i][j], j);
                            // (a logit of infinity has no gradient: 0 times the largest number)
                            dA[j] += out[j] * __builtin_amdgcn_fmed3f(z[i][j], -FLT_MAX, FLT_MAX);
                        }
                    }
                    if (free.on) Raw4<G>::store(to_g.at(), CH, out); else win.put(to_g.at(), out);
                }
                if (!free.on && (first >> i & 1) && p.dh0 && win.n > 0)
                    Raw4<float>::store(p.dh0 + (size_t)m.first[run * RUN + i] * p.C + c, win.n, e);
            }
            to_x.down();
            to_g.down();
        }
    };
    __builtin_amdgcn_s_setprio(0);
    if (plain) finish(Yes{}); else finish(No{});
    if (GATED && p.dA) {                                    // the segment's part of dA: runs in their order
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

// Clears the hand-over's memory (no pair is there yet; tickets and flag 0) and copies states that the call overwrites.
__global__ __launch_bounds__(256) void scan_clear_kernel(ScanChain k, const float *from, float *to, size_t states)
{
    const size_t step = (size_t)gridDim.x * 256, at = (size_t)blockIdx.x * 256 + threadIdx.x;
    for (size_t i = at; i < k.words; i += step) k.part[i] = ~(uint64_t)0;
    for (size_t i = at; i < k.counters; i += step) k.tickets[i] = 0;
    for (size_t i = at; i < states; i += step) to[i] = from[i];
}

// More than SCAN_MANY sequences: those without rows keep their state.  A wave a sequence.
__global__ __launch_bounds__(256) void scan_empty_kernel(const ScanParams p, const float *from, float *to)
{
    for (size_t s = (size_t)blockIdx.x * 4 + threadIdx.x / 64; s < (size_t)p.N; s += (size_t)gridDim.x * 4) {
        int a, b;
        sequence_of(p, (int)s, &a, &b);
        if (b > a) continue;
        for (int c = threadIdx.x % 64; c < p.C; c += 64) to[s * p.C + c] = from ? from[s * p.C + c] : 0.f;
    }
}

// Sums of the segments' parts, in their order: 4.7 us for 128 x 4096.
__global__ __launch_bounds__(256) void scan_sum_kernel(const float *part, int parts, int C, float *out)
{
    __shared__ double s_part[16][16];
    const double sum = column_sum<16>(part, parts, C, s_part);
    const int c = blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x < 16 && c < C) out[c] = (float)sum;
}

// One token a sequence: 8 channels a lane, so that a lane's loads are 16 and 32 bytes.  Bound by memory and by the latency of
// two dependent reads, the slot's and its state's: 512 x 8192 12.0 us (58 MB, 4.8 TB/s), 3 x 2048 3.2 us.
// Slots as for kda_linear_recurrent_step.
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
        const bool complement = p.complement;
        Raw8<T> x;
        Raw8<G> g;
        float A[8];
        x.load((const T *)p.x.p + n * p.x.stride + c, cnt);
        g.load((const G *)p.g.p + n * p.g.stride + c, cnt);
        load_f8(p.state + (size_t)slot * p.C + c, cnt, h);
        if (p.A_log) load_f8(p.A_log + c, cnt, A);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Decay d = decay_of(p.A_log ? p.g_min * sigmoid2(__expf(A[i]) * g[i]).s : not_above_0(g[i]));
            h[i] = decay_step(d, h[i], x[i], complement);
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
    hipLaunchKernelGGL(scan_clear_kernel, dim3((unsigned)(grid < 1024 ? grid : 1024)), dim3(256), 0, stream, p.chain, states,
                       p.state_copy, copied);
    return hipGetLastError();
}

static void launch_empty(const ScanParams &p, const float *from, float *to, hipStream_t stream)
{
    if (!p.cu || p.N <= SCAN_MANY || !to) return;
    const int grid = p.N / 4 < 8192 ? p.N / 4 : 8192;
    hipLaunchKernelGGL(scan_empty_kernel, dim3(grid), dim3(256), 0, stream, p, from, to);
}

template <typename T, typename G> static hipError_t launch_fwd_t(ScanParams p, hipStream_t stream)
{
    const dim3 grid((unsigned)p.chain.segments * ((p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS));
    const hipError_t e = launch_clear(p, p.h0, stream);
    if (e != hipSuccess) return e;
    if (p.state_copy) p.h0 = p.state_copy;
    const auto kernel = p.A_log ? p.chain.words ? scan_fwd_kernel<T, G, true, true> : scan_fwd_kernel<T, G, true, false>
                                : p.chain.words ? scan_fwd_kernel<T, G, false, true> : scan_fwd_kernel<T, G, false, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
    launch_empty(p, p.h0, p.hT, stream);
    return hipGetLastError();
}

template <typename T, typename G> static hipError_t launch_bwd_t(ScanParams p, hipStream_t stream)
{
    const dim3 grid((unsigned)p.chain.segments * ((p.C + SCAN_CHANNELS - 1) / SCAN_CHANNELS));
    const hipError_t e = launch_clear(p, p.dhT, stream);
    if (e != hipSuccess) return e;
    if (p.state_copy) p.dhT = p.state_copy;
    const bool packed = p.hs.scales, both = !p.dg || !p.complement || packed == (p.x.scales != nullptr);
    const auto kernel = p.A_log ? !p.chain.words   ? scan_bwd_kernel<T, G, true, false, EITHER>
                                  : !both          ? scan_bwd_kernel<T, G, true, true, EITHER>
                                  : packed         ? scan_bwd_kernel<T, G, true, true, CODES>
                                                   : scan_bwd_kernel<T, G, true, true, ELEMENTS>
                        : !p.chain.words ? scan_bwd_kernel<T, G, false, false, EITHER>
                        : !both          ? scan_bwd_kernel<T, G, false, true, EITHER>
                        : packed         ? scan_bwd_kernel<T, G, false, true, CODES>
                                         : scan_bwd_kernel<T, G, false, true, ELEMENTS>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
    launch_empty(p, p.dhT, p.dh0, stream);
    if (p.dA)
        hipLaunchKernelGGL(scan_sum_kernel, dim3((p.C + 15) / 16), dim3(256), 0, stream, p.dA_part, p.chain.segments, p.C, p.dA);
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

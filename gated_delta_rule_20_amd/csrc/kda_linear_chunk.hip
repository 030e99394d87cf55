// kda_linear_chunk.hip -- linear attention with a decay per head over whole
// sequences, forward and backward, in the chunkwise-parallel form.
//
// With G the inclusive sum of log-decays inside a chunk, D_rs = e^{G_r - G_s} for s <= r,
// and S the state that enters the chunk:
//   O      = scale * ((Q K^T . D) V + e^G . (Q S))
//   S_next = e^{G_end} S + (e^{G_end - G} . K)^T V
// The gradients are the same product with other operands.  dQ walks the chunks
// forwards with (dO, V, K) in place of (Q, K, V) and the state transposed:
//   dQ = scale * ((dO V^T . D) K + e^G . (dO S^T))
// dV and dK walk them backwards (D_rs = e^{G_s - G_r} for s >= r) with (K, Q, dO) and
// (V, dO, Q), carrying dS, the gradient of the state that leaves the chunk:
//   dV = scale * (K Q^T . D) dO + e^{G_end - G} . (K dS),  dK = scale * (V dO^T . D) Q + e^{G_end - G} . (V dS^T)
//   dS_prev = e^{G_end} dS + scale * (e^G . Q)^T dO
// so one set of building blocks with an operand "Q" of the output rows r, an
// operand "K" of the source rows s, the values "V" and a state [rows of K, columns of V] serves
// all of them.
//
// The decay of a token pair is formed from differences of G held as two floats
// (sum in float64), so it neither overflows nor loses its small value next to a
// large |G|; it is at most 1.
//
// A sequence is walked in order by one workgroup with the state in registers,
// so its traffic is its inputs and outputs.  Where sequences are few, they are
// cut into segments: a first pass walks every segment from a zero state (reading
// K and V only) and leaves its contribution; the second starts each segment from
// the sum of those before it.  That trades half again the traffic for as many workgroups as
// the chip holds.
//
// Roundings: operands of the matrix cores are bf16 for bf16 inputs.  What the state adds
// (decayed V) enters as three bf16 terms, which together hold all 24 bits, so states are exact to
// float32 over any length; the decayed scores and the state as an operand of the outputs are rounded
// once to bf16, as the output is.  The state as an operand of dg's terms keeps three terms too.
#include <type_traits>

#include "kda_common.h"
#include "kda_linear.h"

namespace kda {

template <typename T> constexpr int chunk_of = sizeof(T) == 2 ? 64 : 32;  // tokens per chunk
// LDS row lengths: 32 bytes (bf16) or 16 bytes (fp32) of padding keep the transposing and the row reads off
// one another's banks.
template <typename T> __host__ __device__ constexpr int ld_of(int d) { return d + (sizeof(T) == 2 ? 16 : 4); }
template <typename T> constexpr int ldp_of = chunk_of<T> + 4;
template <typename T> constexpr int split_of = sizeof(T) == 2 ? 3 : 1;    // operand terms that hold a float32

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Fragment whose k-axis is the rows of a row-major LDS tile: value e of lane
// (x, g) is tile[k0 + kmap(g, e)][base + step * (x / 4) + x % 4].  bf16 uses the
// transposing LDS read: each lane names 4 elements of a row, and lane x of a 16-lane group receives column x of
// the 4 x 16 block the group named.
__device__ __forceinline__ bf16x8 col_frag(const bf16 *tile, int ld, int k0, int base, int step)
{
    const int l = lane_id(), x = l & 15, g = l >> 4;
    typedef __attribute__((address_space(3))) bf16x4 *lds_ptr;
    const bf16 *p = tile + (k0 + 4 * g + (x >> 2)) * ld + base + step * (x & 3);
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_ptr)p);
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_ptr)(p + 16 * ld));
    bf16x8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[i] = lo[i]; f[4 + i] = hi[i]; }
    return f;
}
__device__ __forceinline__ f32x8 col_frag(const float *tile, int ld, int k0, int base, int step)
{
    const int l = lane_id(), x = l & 15, g = l >> 4;
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = tile[(k0 + kmap(g, e)) * ld + base + step * (x >> 2) + (x & 3)];
    return f;
}

// x as a sum of NS operand fragments.  Two values at a time: one conversion, then
// their bf16 bits, moved up, are the floats to take off.
template <int NS> __device__ __forceinline__ void split(const float *x, bf16x8 *f)
{
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    typedef float fpair __attribute__((ext_vector_type(2)));
    u32x4 u[NS];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const unsigned w = __builtin_bit_cast(unsigned, __builtin_convertvector((fpair{a, b}), pair));
            u[n][j] = w;
            if (n + 1 < NS) {
                a -= __builtin_bit_cast(float, w << 16);
                b -= __builtin_bit_cast(float, w & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) f[n] = __builtin_bit_cast(bf16x8, u[n]);
}
template <int NS> __device__ __forceinline__ void split(const float *x, f32x8 *f)
{
    static_assert(NS == 1, "float operands need no terms");
#pragma unroll
    for (int e = 0; e < 8; ++e) f[0][e] = x[e];
}

// Global memory is reached through buffer descriptors over uniform bases: a lane
// then holds one 32-bit offset instead of 64-bit addresses (which were spilled, and a reload
// from scratch waits for every load in flight), and rows behind a chunk's last are read as zero
// and not written by the descriptor's bound.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void *base, unsigned bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, bytes, 0x00020000);
}
// n >= 1 rows of `width` bytes, `stride` bytes apart
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_window(const void *base, int n, unsigned stride, unsigned width)
{
    return window(base, (unsigned)(n - 1) * stride + width);
}
__device__ __forceinline__ f32x4 load16(__amdgpu_buffer_rsrc_t rs, int voff, int soff = 0)
{
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, voff, soff, 0));
}
__device__ __forceinline__ bf16x4 load_quad(const bf16 *, __amdgpu_buffer_rsrc_t rs, int voff)
{
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_raw_buffer_load_b64(rs, voff, 0, 0));
}
__device__ __forceinline__ f32x4 load_quad(const float *, __amdgpu_buffer_rsrc_t rs, int voff) { return load16(rs, voff); }
// 4 or 8 neighbouring elements
template <typename T> __device__ __forceinline__ void load_cols(const T *p, __amdgpu_buffer_rsrc_t rs, int voff, quad_t<T> (&v)[1])
{
    v[0] = load_quad(p, rs, voff);
}
__device__ __forceinline__ void load_cols(const bf16 *, __amdgpu_buffer_rsrc_t rs, int voff, bf16x4 (&v)[2])
{
    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(rs, voff, 0, 0);
    v[0] = __builtin_bit_cast(bf16x4, u32x2{w[0], w[1]});
    v[1] = __builtin_bit_cast(bf16x4, u32x2{w[2], w[3]});
}
__device__ __forceinline__ void load_cols(const float *, __amdgpu_buffer_rsrc_t rs, int voff, f32x4 (&v)[2])
{
    v[0] = load16(rs, voff);
    v[1] = load16(rs, voff + 16);
}
__device__ __forceinline__ void store_quad(__amdgpu_buffer_rsrc_t rs, int voff, bf16x4 v)
{
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), rs, voff, 0, 0);
}
__device__ __forceinline__ void store_quad(__amdgpu_buffer_rsrc_t rs, int voff, f32x4 v, int soff = 0)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, voff, soff, 0);
}
__device__ __forceinline__ void store_oct(__amdgpu_buffer_rsrc_t rs, int voff, bf16x8 v)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, voff, 0, 0);
}
__device__ __forceinline__ void store_oct(__amdgpu_buffer_rsrc_t rs, int voff, f32x8 v)
{
    store_quad(rs, voff, f32x4{v[0], v[1], v[2], v[3]});
    store_quad(rs, voff + 16, f32x4{v[4], v[5], v[6], v[7]});
}

// One chunk tile [C][D] on its way from global memory to LDS, NT threads.
template <typename T, int D, int NT> struct Stage {
    static constexpr int C = chunk_of<T>, ROW = D * (int)sizeof(T) / 16, N = C * ROW / NT;
    static_assert(N * NT == C * ROW && NT % ROW == 0, "tile divides evenly");
    f32x4 r[N];
    // rows [0, n) of base (n >= 1), `stride` elements apart; the others are zero
    __device__ __forceinline__ void load(const T *base, size_t stride, int n, int t)
    {
        const unsigned sb = (unsigned)(stride * sizeof(T));
        const __amdgpu_buffer_rsrc_t rs = rows_window(base, n, sb, D * sizeof(T));
        const unsigned at = (unsigned)(t / ROW) * sb + (unsigned)(t % ROW) * 16;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = load16(rs, (int)(at + (unsigned)(i * (NT / ROW)) * sb));
    }
    __device__ __forceinline__ void store(T *tile, int t) const
    {
        char *p = (char *)tile + (t / ROW) * (ld_of<T>(D) * (int)sizeof(T)) + (t % ROW) * 16;
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<f32x4 *>(p + i * (NT / ROW) * (ld_of<T>(D) * (int)sizeof(T))) = r[i];
    }
};

// Decay vectors of one chunk.
template <int C> struct alignas(16) Decay {
    float hi[C], lo[C];      // G in units of log 2, as hi + lo
    float inter[C];          // factor of the state's part of output row r
    float state[C];          // factor of source row s in the state
    float total;             // e^{G_end}
};

// One wave: lane u holds the log-decay of token u (0 behind the chunk's last).
template <int C, bool REV> __device__ __forceinline__ void make_decay(Decay<C> *d, float x, float scale)
{
    const int u = lane_id();
    double G = u < C ? (double)log2_decay(x) : 0.0;
#pragma unroll
    for (int s = 1; s < C; s *= 2) {
        const double y = __shfl_up(G, s);
        if (u >= s) G += y;
    }
    const double end = __shfl(G, C - 1);
    const float in = __builtin_amdgcn_exp2f((float)G), out = __builtin_amdgcn_exp2f((float)(end - G));
    if (u < C) {
        const float hi = (float)G;
        d->hi[u] = hi;
        d->lo[u] = (float)(G - (double)hi);
        d->inter[u] = REV ? out : scale * in;
        d->state[u] = REV ? scale * in : out;
    }
    if (u == C - 1) d->total = in;
}

// The sum over the 16 lanes of a row, in each of them.
__device__ __forceinline__ float row_total(float v)
{
    v = dpp_add<0xB1, 0xF>(v);   // quad_perm [1, 0, 3, 2]
    v = dpp_add<0x4E, 0xF>(v);   // quad_perm [2, 3, 0, 1]
    v = dpp_add<0x141, 0xF>(v);  // row_half_mirror
    return dpp_add<0x140, 0xF>(v);  // row_mirror
}

// Sums over a row's 16 lanes from this one on, and over those before it.
__device__ __forceinline__ float row_from(float v)
{
    v = dpp_add<0x101, 0xF>(v);  // row_shl:1, 2, 4, 8; nothing comes in from outside the row
    v = dpp_add<0x102, 0xF>(v);
    v = dpp_add<0x104, 0xF>(v);
    return dpp_add<0x108, 0xF>(v);
}
__device__ __forceinline__ float row_before(float v)
{
    v = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x111, 0xF, 0xF, false));
    v = dpp_add<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    return dpp_add<0x118, 0xF>(v);
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ double wave_total(double v)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
    return v;
}

// The work of NW = 4 waves on one chunk: output columns (and state columns) are
// dealt 16 * NCT to a wave.  DK: contracted width, DV: output width.
constexpr int NW = 4;
template <typename T, int DK, int DV, bool REV> struct Group {
    static constexpr int C = chunk_of<T>, NT = C / 16, NRT = DK / 16, NCT = DV / 16 / NW, KS = DK / 32, CK = C / 32;
    static constexpr int LDK = ld_of<T>(DK), LDV = ld_of<T>(DV), LDP = ldp_of<T>;

    // With two column tiles a lane's rows of both tiles are made neighbours (8 columns: one wide access).
    static __device__ __forceinline__ int col0(int w, int ct) { return NCT == 2 ? 32 * w + 4 * ct : 16 * w; }
    static constexpr int STEP = NCT == 2 ? 8 : 4;

    // ---- state, accumulator layout: value i of lane (x, g) in tile [rt][ct] is S[row(rt) + 8 g + i][column x of ct].
    // Rows are dealt so that the tiles 2 ks and 2 ks + 1 hold, in one lane, the rows 32 ks + 8 g .. + 7: as an
    // operand of the outputs they meet 8 neighbouring elements of a row of Q, one 16-byte read free of bank
    // conflicts (two 8-byte reads of the common deal were four-way conflicts).
    static constexpr __device__ int row(int rt) { return 32 * (rt >> 1) + 4 * (rt & 1); }
    f32x4 S[NRT][NCT];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) S[rt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // m in memory as [DK][DV], or [DV][DK] when TR: this lane's offset, and tile (rt, ct)'s row i from there
    template <bool TR> static __device__ __forceinline__ int state_lane(int w)
    {
        const int l = lane_id(), x = l & 15, g = l >> 4, col = col0(w, 0) + STEP * (x >> 2) + (x & 3);
        return 4 * (TR ? col * DK + 8 * g : 8 * g * DV + col);
    }
    template <bool TR> static constexpr __device__ int state_at(int rt, int ct, int i)
    {
        return 4 * (TR ? 4 * ct * DK + row(rt) : (row(rt) + i) * DV + 4 * ct);
    }
    template <bool TR> static __device__ __forceinline__ f32x4 fetch(__amdgpu_buffer_rsrc_t m, int at, int rt, int ct)
    {
        if (TR) return load16(m, at, state_at<TR>(rt, ct, 0));
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(m, at, state_at<TR>(rt, ct, i), 0));
        return v;
    }
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t state_window(const float *m) { return window(m, DK * DV * 4); }

    // S = f * S + m
    template <bool TR> __device__ __forceinline__ void add(const float *m, float f, int w)
    {
        const __amdgpu_buffer_rsrc_t rs = state_window(m);
        const int at = state_lane<TR>(w);
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) S[rt][ct] = S[rt][ct] * f + fetch<TR>(rs, at, rt, ct);
    }
    // The same for a state kept in the order of the registers (parts, read by workgroups of the same geometry):
    // a wave's access is 1 KiB in a row.
    __device__ __forceinline__ void add_part(const float *m, float f, int w)
    {
        const __amdgpu_buffer_rsrc_t rs = state_window(m);
        const int at = 16 * (64 * w + lane_id());
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) S[rt][ct] = S[rt][ct] * f + load16(rs, at, 1024 * NW * (rt * NCT + ct));
    }
    __device__ __forceinline__ void put_part(float *m, int w) const
    {
        const __amdgpu_buffer_rsrc_t rs = state_window(m);
        const int at = 16 * (64 * w + lane_id());
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) store_quad(rs, at, S[rt][ct], 1024 * NW * (rt * NCT + ct));
    }
    template <bool TR> __device__ __forceinline__ void put(float *m, int w) const
    {
        const __amdgpu_buffer_rsrc_t rs = state_window(m);
        const int at = state_lane<TR>(w);
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                if (TR)
                    store_quad(rs, at, S[rt][ct], state_at<TR>(rt, ct, 0));
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = S[rt][ct][i];          // (a vector's element cannot be bit-cast in place)
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), rs, at,
                                                              state_at<TR>(rt, ct, i), 0);
                    }
            }
    }
    template <bool TR> __device__ __forceinline__ double dot(const float *m, int w) const
    {
        const __amdgpu_buffer_rsrc_t rs = state_window(m);
        const int at = state_lane<TR>(w);
        f32x4 y[NRT][NCT];
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) y[rt][ct] = fetch<TR>(rs, at, rt, ct);
        __builtin_amdgcn_sched_barrier(0);                     // one wait for all of it
        double s = 0.0;
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) s += (double)S[rt][ct][i] * (double)y[rt][ct][i];
        return wave_total(s);
    }

    // The chunk's addition to the state.
    __device__ __forceinline__ void update(const T *K, const T *V, const Decay<C> &d, int w)
    {
        constexpr int NS = split_of<T>;
        const int g = lane_id() >> 4;
        const float f = d.total;
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) S[rt][ct] *= f;
#pragma unroll
        for (int ks = 0; ks < CK; ++ks) {
            frag_t<T> vf[NCT][NS];
            const f32x4 a = *reinterpret_cast<const f32x4 *>(&d.state[32 * ks + 4 * g]);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(&d.state[32 * ks + 16 + 4 * g]);
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const frag_t<T> v = col_frag(V, LDV, 32 * ks, col0(w, ct), STEP);
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) { x[e] = to_f<T>(v[e]) * a[e]; x[4 + e] = to_f<T>(v[4 + e]) * b[e]; }
                split<NS>(x, vf[ct]);
            }
#pragma unroll
            for (int rt = 0; rt < NRT; ++rt) {
                const frag_t<T> kf = col_frag(K, LDK, 32 * ks, row(rt), 8);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int n = 0; n < NS; ++n) S[rt][ct] = mma(kf, vf[ct][n], S[rt][ct]);
                if (rt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    // Raw scores of tile (source rows st, output rows rt): value i of lane (x, g) belongs to s = 16 st + 4 g + i, r = 16 rt + x.
    static __device__ __forceinline__ f32x4 scores(const T *Q, const T *K, int rt, int st)
    {
        const int l = lane_id(), x = l & 15, g = l >> 4;
        frag_t<T> k[KS], q[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            k[ks] = load_frag_lin<T>(K + (16 * st + x) * LDK + 32 * ks, g);
            q[ks] = load_frag_lin<T>(Q + (16 * rt + x) * LDK + 32 * ks, g);
        }
        __builtin_amdgcn_sched_barrier(0);                     // all reads in flight before the first product
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) acc = mma(k[ks], q[ks], acc);
        return acc;
    }
    // Those scores with their decays, 0 where s is not a source of r (on the diagonal tile).
    static __device__ __forceinline__ f32x4 decayed(f32x4 p, const Decay<C> &d, float scale, int rt, int st)
    {
        const int l = lane_id(), x = l & 15, g = l >> 4;
        const int r = 16 * rt + x, s = 16 * st + 4 * g;
        const float rh = d.hi[r], rl = d.lo[r];
        const f32x4 sh = *reinterpret_cast<const f32x4 *>(&d.hi[s]), sl = *reinterpret_cast<const f32x4 *>(&d.lo[s]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float y = REV ? (sh[i] - rh) + (sl[i] - rl) : (rh - sh[i]) + (rl - sl[i]);
            p[i] *= scale * __builtin_amdgcn_exp2f(y);
        }
        if (rt == st) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = (REV ? 4 * g + i >= x : 4 * g + i <= x) ? p[i] : 0.f;
        }
        return p;
    }
    static __device__ __forceinline__ void put_scores(T *P, f32x4 p, int rt, int st)
    {
        const int l = lane_id(), x = l & 15, g = l >> 4;
        *reinterpret_cast<quad_t<T> *>(P + (16 * rt + x) * LDP + 16 * st + 4 * g) = make_quad<T>(p);
    }
    static constexpr __device__ bool reached(int rt, int st) { return REV ? st >= rt : st <= rt; }

    // P's tiles that no source reaches but that a product takes in with its 32 source rows: zero, once.
    static __device__ __forceinline__ void clear_scores(T *P, int w)
    {
        if (w < NT / 2) put_scores(P, f32x4{0.f, 0.f, 0.f, 0.f}, REV ? 2 * w + 1 : 2 * w, REV ? 2 * w : 2 * w + 1);
    }

    // Decayed scores into P[r][s] (rounded to T).  Of the ten tiles of a 64-token chunk each of three waves takes three:
    // (0,0) (3,0) (3,1), (1,0) (1,1) (3,2) and (2,0) (2,1) (2,2), and the fourth takes (3,3) and the next chunk's
    // decays; backwards all is mirrored.  Of a 32-token chunk's three tiles each wave takes one.
    static __device__ __forceinline__ void make_scores(T *P, const T *Q, const T *K, const Decay<C> &d, float scale, int w)
    {
        for_tiles(w, [&](int rt, int st) { put_scores(P, decayed(scores(Q, K, rt, st), d, scale, rt, st), rt, st); });
    }
    template <typename F> static __device__ __forceinline__ void for_tiles(int w, F f)
    {
#pragma unroll
        for (int i = 0; i < (NT == 4 ? 3 : 1); ++i) {
            int rt, st;
            if (NT == 4) {
                if (w == 3 && i > 0) break;
                rt = w == 3 ? 3 : w == 2 ? 2 : w == 1 ? (i < 2 ? 1 : 3) : (i < 1 ? 0 : 3);
                st = w == 3 ? 3 : w == 2 ? i : w == 1 ? i : (i < 1 ? 0 : i - 1);
            } else {
                if (w >= 3) break;
                rt = w > 0;
                st = w > 1;
            }
            if (REV) { rt = NT - 1 - rt; st = NT - 1 - st; }
            f(rt, st);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The state's part of the outputs: O[it][ct], value i of lane (x, g) is output column 4 g + i of ct, row 16 it + x.
    template <int NS> __device__ __forceinline__ void inter(f32x4 (&O)[NT][NCT], const T *Q, const Decay<C> &d) const
    {
        const int l = lane_id(), x = l & 15, g = l >> 4;
#pragma unroll
        for (int it = 0; it < NT; ++it)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) O[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            frag_t<T> sf[NCT][NS];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) { y[e] = S[2 * ks][ct][e]; y[4 + e] = S[2 * ks + 1][ct][e]; }
                split<NS>(y, sf[ct]);
            }
#pragma unroll
            for (int it = 0; it < NT; ++it) {
                const frag_t<T> qf = load_frag_lin<T>(Q + (16 * it + x) * LDK + 32 * ks, g);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int n = 0; n < NS; ++n) O[it][ct] = mma(sf[ct][n], qf, O[it][ct]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int it = 0; it < NT; ++it) {
            const float f = d.inter[16 * it + x];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) O[it][ct] *= f;
        }
    }

    // The chunk's own part of the outputs.
    static __device__ __forceinline__ void intra(f32x4 (&O)[NT][NCT], const T *P, const T *V, int w)
    {
        const int l = lane_id(), x = l & 15, g = l >> 4;
#pragma unroll
        for (int ks = 0; ks < CK; ++ks) {
            frag_t<T> vf[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) vf[ct] = col_frag(V, LDV, 32 * ks, col0(w, ct), STEP);
#pragma unroll
            for (int it = 0; it < NT; ++it) {
                if (!(reached(it, 2 * ks) || reached(it, 2 * ks + 1))) continue;
                const frag_t<T> pf = load_frag_kmap<T>(P + (16 * it + x) * LDP + 32 * ks, g);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) O[it][ct] = mma(vf[ct], pf, O[it][ct]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // A lane's output columns of row 16 it + x, from `first` on.
    static __device__ __forceinline__ int first_col(int w)
    {
        const int g = lane_id() >> 4;
        return NCT == 2 ? 32 * w + 8 * g : 16 * w + 4 * g;
    }
    template <typename U>
    static __device__ __forceinline__ void store(U *o, size_t stride, int n, const f32x4 (&O)[NT][NCT], int w)
    {
        const int x = lane_id() & 15;
        const unsigned sb = (unsigned)(stride * sizeof(U));
        const __amdgpu_buffer_rsrc_t rs = rows_window(o, n, sb, DV * sizeof(U));
        const unsigned at = (unsigned)x * sb + first_col(w) * (unsigned)sizeof(U);
#pragma unroll
        for (int it = 0; it < NT; ++it) {
            const int p = (int)(at + 16u * it * sb);
            if constexpr (NCT == 2) {
                const float y[8] = {O[it][0][0], O[it][0][1], O[it][0][2], O[it][0][3],
                                    O[it][1][0], O[it][1][1], O[it][1][2], O[it][1][3]};
                store_oct(rs, p, make_frag<U>(y));
            } else {
                store_quad(rs, p, make_quad<U>(O[it][0]));
            }
        }
    }
    // For each row 16 it + x: the sum over this wave's columns of O times m's row; m in LDS, or in global memory
    // (n rows, `stride` elements apart) through `quads`.
    template <typename F>
    static __device__ __forceinline__ void row_dots(float *out, F quads, const f32x4 (&O)[NT][NCT])
    {
        const int l = lane_id(), x = l & 15, g = l >> 4;
#pragma unroll
        for (int it = 0; it < NT; ++it) {
            float s = 0.f;
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const f32x4 y = quad_to_f<T>(quads(it, ct));
#pragma unroll
                for (int i = 0; i < 4; ++i) s += O[it][ct][i] * y[i];
            }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (g == 0) out[16 * it + x] = s;
        }
    }
};

// ---- which tokens a workgroup walks ----------------------------------------------------------------------------------

struct Piece {
    int seq, part, parts;     // segment `part` of the sequence's `parts`
    int begin, len;           // the sequence's first row and its tokens
    int slot, anchor;         // index of the sequence's first part in the workspace, and of its first anchor
};

// Segment `id` of all sequences' segments of L tokens (an empty sequence has
// one), sequence by sequence; false when there are fewer.  A sequence of n
// segments has n - 1 parts in the workspace (nothing is left by its last one, or
// first one backwards).  Every wave finds the segment by itself: 64
// sequences at a time, a prefix sum over the lanes.  L and LA are at least 128, so the sums fit 32 bits unsigned.
__device__ __forceinline__ int pieces_of(int len, int L) { return len <= 0 ? 1 : (len - 1) / L + 1; }

__device__ __forceinline__ bool find_piece(const LinearChunkParams &p, int id, Piece &w)
{
    const int L = p.seg, LA = p.anchor_tokens;
    if (!p.cu) {
        w.parts = pieces_of(p.T, L);
        w.seq = id / w.parts;
        w.part = id % w.parts;
        w.begin = w.seq * p.T;
        w.len = p.T;
        w.slot = w.seq * (w.parts - 1);
        w.anchor = w.seq * (pieces_of(p.T, LA) - 1);
        return w.seq < p.N;
    }
    if (p.seq_of) {
        const int s = p.seq_of[id];
        if (s < 0) return false;
        const int a = min(max(p.cu[s], 0), p.T);
        w.seq = s;
        w.begin = a;
        w.len = min(max(p.cu[s + 1], a), p.T) - a;
        w.parts = pieces_of(w.len, L);
        w.part = id - p.first_seg[s];
        w.slot = p.first_seg[s] - s;
        w.anchor = p.first_anchor[s] - s;
        return true;
    }
    const int lane = lane_id();
    unsigned before = 0, abefore = 0;
    for (int s0 = 0; s0 < p.N; s0 += 64) {
        const int s = s0 + lane;
        int a = 0, b = 0, n = 0, na = 0;
        if (s < p.N) {
            a = min(max(p.cu[s], 0), p.T);
            b = min(max(p.cu[s + 1], a), p.T);
            n = pieces_of(b - a, L);
            na = pieces_of(b - a, LA);
        }
        unsigned x = n, y = na;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const unsigned u = __shfl_up(x, d), v = __shfl_up(y, d);
            if (lane >= d) { x += u; y += v; }
        }
        const unsigned long long over = __ballot(before + x > (unsigned)id);
        if (over) {
            const int f = __ffsll(over) - 1;
            w.seq = s0 + f;
            w.parts = __builtin_amdgcn_readlane(n, f);
            w.part = (int)((unsigned)id - before - (__builtin_amdgcn_readlane(x, f) - (unsigned)w.parts));
            w.begin = __builtin_amdgcn_readlane(a, f);
            w.len = __builtin_amdgcn_readlane(b, f) - w.begin;
            w.slot = id - w.part - w.seq;
            w.anchor = (int)(abefore + __builtin_amdgcn_readlane(y, f) - __builtin_amdgcn_readlane(na, f)) - w.seq;
            return true;
        }
        before += __builtin_amdgcn_readlane(x, 63);
        abefore += __builtin_amdgcn_readlane(y, 63);
    }
    return false;
}

// The parts of sequence s, of a few: the index of the first and their number.
__device__ __forceinline__ void parts_of(const LinearChunkParams &p, int s, int &slot, int &n)
{
    if (!p.cu) {
        n = pieces_of(p.T, p.seg) - 1;
        slot = s * n;
        return;
    }
    const auto parts = [&](int i) {
        const int a = min(max(p.cu[i], 0), p.T), b = min(max(p.cu[i + 1], a), p.T);
        return pieces_of(b - a, p.seg) - 1;
    };
    n = parts(s);
    long before = 0;
    for (int i = 0; i < s; ++i) before += parts(i);
    slot = (int)min(before, 0x7fffffffL);
}

// One workgroup: the tables of find_piece for many sequences.  Sums in 64 bits, so
// that offsets that break the rules cannot wrap; what lies beyond n_seg is cut off.
__global__ __launch_bounds__(1024) void linear_table_kernel(const LinearChunkParams p)
{
    __shared__ unsigned long long s_seg[16], s_anchor[16];
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
    unsigned long long segs = 0, anchors = 0;
    for (int s0 = 0; s0 < p.N; s0 += 1024) {
        const int s = s0 + t;
        int n = 0, na = 0;
        if (s < p.N) {
            const int a = min(max(p.cu[s], 0), p.T), b = min(max(p.cu[s + 1], a), p.T);
            n = pieces_of(b - a, p.seg);
            na = pieces_of(b - a, p.anchor_tokens);
        }
        unsigned long long x = n, y = na;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const unsigned long long u = __shfl_up(x, d), v = __shfl_up(y, d);
            if (lane >= d) { x += u; y += v; }
        }
        if (lane == 63) { s_seg[wv] = x; s_anchor[wv] = y; }
        __syncthreads();
        unsigned long long first = segs + x - n, afirst = anchors + y - na;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < wv) { first += s_seg[i]; afirst += s_anchor[i]; }
            segs += s_seg[i];
            anchors += s_anchor[i];
        }
        __syncthreads();
        if (s < p.N) {
            p.first_seg[s] = (int)min(first, 0x7fffffffull);
            p.first_anchor[s] = (int)min(afirst, 0x7fffffffull);
            for (int i = 0; i < n && first + i < (unsigned long long)p.n_seg; ++i) p.seq_of[first + i] = s;
        }
    }
    for (unsigned long long i = segs + t; i < (unsigned long long)p.n_seg; i += 1024) p.seq_of[i] = -1;
}
static hipError_t launch_table(const LinearChunkParams &p, hipStream_t stream)
{
    if (!p.seq_of) return hipSuccess;
    hipLaunchKernelGGL(linear_table_kernel, dim3(1), dim3(1024), 0, stream, p);
    return hipGetLastError();
}

// Where the state at token `pos` of the sequence is kept for dg, or -1.  Offsets
// that break the rules of cu_seqlens can ask for more than there is room for.
__device__ __forceinline__ long anchor_at(const LinearChunkParams &p, const Piece &w, int pos)
{
    if (pos == w.len) return p.anchor_end ? (long)p.n_anchors + w.seq : -1;
    if (pos % p.anchor_tokens != 0) return -1;
    const long i = (long)w.anchor + pos / p.anchor_tokens - 1;
    return i < p.n_anchors ? i : -1;
}

// Where the entering and the resulting states are one array, other segments of a
// sequence may still read its entry when the segment that forms the result is
// done.  The result then waits in part i of the sequence, which that segment alone reads.
__device__ __forceinline__ bool deferred(const LinearChunkParams &p, const Piece &w, int i)
{
    return p.defer && w.parts > 1 && w.slot + i < p.n_part;
}

// The log-decay of a chunk's token u for this lane, 0 behind the last; as it is in memory, so that nothing waits
// for it here.  n >= 1.
__device__ __forceinline__ float fetch_decay(const LinearChunkParams &p, int row, int h, int n)
{
    const int u = lane_id();
    const unsigned step = 4u * (unsigned)p.H;
    const __amdgpu_buffer_rsrc_t rs = p.g_per_head ? window(p.g + h, 4) : rows_window(p.g + (size_t)row * p.H + h, n, step, 4);
    const unsigned at = !p.g_per_head ? u * step : u < n ? 0u : 4u;
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (int)at, 0, 0));
}

enum { WALK_STATE, WALK_STATE_REV, WALK_OUT, WALK_DQ, WALK_STATE_DQ, WALK_DQ_DG };

// One workgroup walks one segment for one value head (head fastest, so that
// workgroups that run together read neighbouring rows).
//   WALK_STATE      q, k, v roles: -, k, v;  writes the segment's part and decay
//   WALK_STATE_REV  -, q, do, backwards; writes its part in both orders that linear_dkdv_kernel reads
//   WALK_STATE_DQ   -, v, k: as WALK_STATE, transposed (DK = the problem's Dv, DV = its Dk)
//   WALK_OUT        q, k, v;  writes o, final state, checkpoints
//   WALK_DQ         do, v, k (DK = the problem's Dv, DV = its Dk);  writes dq
//   WALK_DQ_DG      the same with y and anchors for dg
// 66 KiB of LDS and up to 256 registers a lane: two workgroups share a compute
// unit, and one computes while the other waits for memory.  Eight waves of half the
// columns each hide more latency but read Q and K from LDS twice as often (133 K packed
// tokens: 1.41 ms against 1.26 ms at the time).
// Measured at H = 32, d = 128, bf16: 64 packed sequences of 128 to 4096 tokens 1.10 ms, 4.66 GB,
// 4.2 TB/s or 86% of a copy: bound by HBM.  T = 8192: 111 us a call; state pass 38 us (3.5 TB/s), output 74 us
// (3.6 TB/s, with up to 15 states summed at the start; matrix cores busy 22% of the time, bank conflicts 17% of the
// LDS cycles).  T = 131072: 1.44 ms for both.
template <typename T, int DK, int DV, int MODE>
__global__ __launch_bounds__(64 * NW, 2) void linear_walk_kernel(const LinearChunkParams p)
{
    constexpr int THREADS = 64 * NW;
    constexpr bool DG = MODE == WALK_DQ_DG, DQ = MODE == WALK_DQ || DG;
    constexpr bool REV = MODE == WALK_STATE_REV, OUT = MODE == WALK_OUT || DQ, TR = DQ;
    using G = Group<T, DK, DV, REV>;
    constexpr int C = G::C;
    __shared__ __align__(16) T sQ[OUT ? C * G::LDK : 8];
    __shared__ __align__(16) T sK[C * G::LDK];
    __shared__ __align__(16) T sV[C * G::LDV];
    __shared__ __align__(16) T sP[OUT ? C * G::LDP : 8];
    __shared__ __align__(16) Decay<C> sD[2];
    __shared__ float sY[DG ? 4 : 1][C];

    const int h = (int)(blockIdx.x % (unsigned)p.H), id = (int)(blockIdx.x / (unsigned)p.H);
    Piece w;
    if (!find_piece(p, id, w)) return;
    if ((MODE == WALK_STATE || MODE == WALK_STATE_DQ) && w.part == w.parts - 1) return;   // nothing comes after it
    if (MODE == WALK_STATE_REV && w.part == 0) return;
    const int slot = w.slot + (MODE == WALK_STATE_REV ? w.part - 1 : w.part);
    if (!OUT && slot >= p.n_part) return;                      // only with offsets that break the rules
    const int t = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(t >> 6);
    const int first = w.part * p.seg, toks = min(p.seg, w.len - first);
    const int nc = (max(toks, 0) + C - 1) / C;
    const int row0 = w.begin + first;
    const int hk = h / p.group, Hk = p.H / p.group;
    // strides and heads of the three roles
    constexpr bool QK_SHARED = !DQ && MODE != WALK_STATE_DQ;    // role q / k carry the query / key heads
    const size_t sq = (size_t)(QK_SHARED ? Hk : p.H) * DK;
    const size_t sv = (size_t)(QK_SHARED ? p.H : Hk) * DV;
    const T *gq = (const T *)p.q + (size_t)(QK_SHARED ? hk : h) * DK;
    const T *gk = (const T *)p.k + (size_t)(QK_SHARED ? hk : h) * DK;
    const T *gv = (const T *)p.v + (size_t)(QK_SHARED ? h : hk) * DV;

    G grp;
    grp.clear();
    const size_t pair = (size_t)w.seq * p.H + h, part_size = (size_t)DK * DV;
    if (OUT) {
        if (p.h0) grp.template add<TR>(p.h0 + pair * part_size, 0.f, wv);
        for (int i = p.summed ? max(w.part - 1, 0) : 0; i < w.part; ++i) {
            if (w.slot + i >= p.n_part) break;
            const size_t at = (size_t)(w.slot + i) * p.H + h;
            grp.add_part(p.part + at * part_size, p.dec[at], wv);
        }
    }
    Stage<T, DK, THREADS> rq, rk;
    Stage<T, DV, THREADS> rv;
    float rg = 0.f, dec = 1.f;
    // the next chunk's rows
    const int chunk0 = row0 + (REV ? max(nc - 1, 0) : 0) * C;
    gq += (size_t)chunk0 * sq;
    gk += (size_t)chunk0 * sq;
    gv += (size_t)chunk0 * sv;
    const long step_q = (REV ? -C : C) * (long)sq, step_v = (REV ? -C : C) * (long)sv;
    auto fetch = [&](int c) {
        const int n = min(C, toks - c * C);
        if (OUT) rq.load(gq, sq, n, t);
        rk.load(gk, sq, n, t);
        rv.load(gv, sv, n, t);
        gq += step_q;
        gk += step_q;
        gv += step_v;
    };
    // decays are fetched two chunks ahead: they are summed while the tiles of the chunk between are in flight
    auto decays_of = [&](int i) {
        const int c = REV ? nc - 1 - i : i;
        return fetch_decay(p, row0 + c * C, h, min(C, toks - c * C));
    };
    if (OUT) G::clear_scores(sP, wv);
    if (nc > 0) {
        fetch(REV ? nc - 1 : 0);
        if (wv == NW - 1) {
            make_decay<C, REV>(&sD[0], decays_of(0), p.scale);
            if (nc > 1) rg = decays_of(1);
        }
    }
    for (int i = 0; i < nc; ++i) {
        const int c = REV ? nc - 1 - i : i, n = min(C, toks - c * C), row = row0 + c * C;
        const Decay<C> &d = sD[i & 1];
        lds_barrier();                                         // the last chunk has been read
        if (OUT) rq.store(sQ, t);
        rk.store(sK, t);
        rv.store(sV, t);
        lds_barrier();
        // q's rows for y, before the next tiles: what is loaded later is waited for later
        quad_t<T> yq[DG ? G::NT : 1][G::NCT];
        if constexpr (DG) {
            const T *q0 = (const T *)p.q_rows + ((size_t)row * Hk + hk) * DV;
            const unsigned sb = (unsigned)(Hk * DV * sizeof(T));
            const __amdgpu_buffer_rsrc_t rs = rows_window(q0, n, sb, DV * sizeof(T));
            const unsigned at = (unsigned)(t & 15) * sb + G::first_col(wv) * (unsigned)sizeof(T);
#pragma unroll
            for (int it = 0; it < G::NT; ++it) load_cols(q0, rs, (int)(at + 16u * it * sb), yq[it]);
        }
        if (!DG && i + 1 < nc) fetch(REV ? c - 1 : c + 1);
        auto next_decay = [&]() {
            if (wv != NW - 1 || i + 1 >= nc) return;
            const float x = rg;
            if (i + 2 < nc) rg = decays_of(i + 2);
            make_decay<C, REV>(&sD[(i + 1) & 1], x, p.scale);
        };
        if constexpr (OUT) {
            f32x4 O[G::NT][G::NCT];
            G::make_scores(sP, sQ, sK, d, p.scale, wv);
            if constexpr (DG) {
                grp.template inter<split_of<T>>(O, sQ, d);
                G::row_dots(sY[wv], [&](int it, int ct) { return yq[it][ct]; }, O);
                if (i + 1 < nc) fetch(c + 1);                  // here, where q's rows have left their registers
            } else {
                grp.template inter<1>(O, sQ, d);
            }
            next_decay();
            lds_barrier();                                     // P (and y) are whole
            G::intra(O, sP, sV, wv);
            if (DQ && p.wide)
                G::store((float *)p.o + ((size_t)row * p.H + h) * DV, (size_t)p.H * DV, n, O, wv);
            else if (DQ)
                G::store((T *)p.o + ((size_t)row * Hk + hk) * DV, (size_t)Hk * DV, n, O, wv);
            else
                G::store((T *)p.o + ((size_t)row * p.H + h) * DV, (size_t)p.H * DV, n, O, wv);
            if (DG && t < n)
                p.y[(size_t)(row + t) * p.H + h] = (sY[0][t] + sY[1 % 4][t]) + (sY[2 % 4][t] + sY[3 % 4][t]);
        } else {
            next_decay();
            dec *= d.total;
        }
        grp.update(sK, sV, d, wv);
        const int pos = first + c * C + n;                     // tokens of the sequence behind this chunk's end
        if (MODE == WALK_OUT && p.ckpt && n == C && pos < w.len) {
            const int every = p.ckpt_every * CHUNK;
            if (pos % every == 0 && pos / every <= p.ckpt_slots)
                grp.template put<TR>(p.ckpt + (((size_t)w.seq * p.ckpt_slots + pos / every - 1) * p.H + h) * part_size, wv);
        }
        if (DG) {
            const long a = anchor_at(p, w, pos);
            if (a >= 0) grp.template put<TR>(p.anchors + ((size_t)a * p.H + h) * part_size, wv);
        }
    }
    if (!OUT) {
        const size_t at = (size_t)slot * p.H + h;
        grp.put_part(p.part + at * part_size, wv);
        if (MODE == WALK_STATE_REV) grp.template put<false>(p.part_tr + at * part_size, wv);
        if (t == 0) p.dec[at] = dec;
    }
    if (MODE == WALK_OUT && p.hT && w.part == w.parts - 1)
        grp.template put<TR>(deferred(p, w, w.parts - 2) ? p.part + ((size_t)(w.slot + w.parts - 2) * p.H + h) * part_size
                                                         : p.hT + pair * part_size, wv);
}

// The states that linear_walk_kernel (backwards: linear_dkdv_kernel) deferred, to their place.
__global__ __launch_bounds__(256) void linear_deferred_kernel(const LinearChunkParams p, float *out, int backwards, int state)
{
    const int h = (int)(blockIdx.x % (unsigned)p.H), id = (int)(blockIdx.x / (unsigned)p.H);
    Piece w;
    if (!find_piece(p, id, w) || w.part != 0) return;
    const int i = backwards ? 0 : w.parts - 2;
    if (!deferred(p, w, i)) return;
    const f32x4 *src = reinterpret_cast<const f32x4 *>(p.part + ((size_t)(w.slot + i) * p.H + h) * state);
    f32x4 *dst = reinterpret_cast<f32x4 *>(out + ((size_t)w.seq * p.H + h) * state);
    for (int e = threadIdx.x; e < state / 4; e += 256) dst[e] = src[e];
}

// Sums of the parts in place, so that a segment of the backward walks starts from
// one state and one decay: part i becomes what all of the sequence's parts up to i
// (backwards: from i on) leave at its end.  For calls of at most 16 (sequence, head)
// pairs with more than 6 segments to a sequence, where a segment's own sum of up to n
// states is the longer path (whole backward, bf16, D = 128): T = 1024, H = 4: 73 -> 62
// us, T = 4096, H = 8: 135 -> 99, T = 8192, H = 2: 177 -> 108, T = 16384, H = 16:
// 414 -> 370.  With more pairs the segments' own sums hide behind one another's
// products, and a launch more costs (H = 32: T = 1024 85 -> 91, T = 4096 193 -> 200).
// blockIdx.x: the pair; .y: which array; .z: 1024 elements of the state.
__global__ __launch_bounds__(256) void linear_scan_kernel(const LinearBwdParams b, int state)
{
    const LinearChunkParams &p = b.c;
    const bool forwards = blockIdx.y == 0;
    float *part = forwards ? b.part_fwd : blockIdx.y == 1 ? p.part : p.part_tr;
    const float *dec = forwards ? b.dec_fwd : p.dec;
    float *sum = forwards ? b.sum_fwd : b.sum_rev;
    const bool scribe = blockIdx.z == 0 && blockIdx.y < 2 && threadIdx.x == 0;
    const size_t e = (size_t)blockIdx.z * 1024 + threadIdx.x * 4;
    const int h = (int)(blockIdx.x % p.H);
    int slot, n;
    parts_of(p, (int)(blockIdx.x / p.H), slot, n);
    n = min(n, p.n_part - slot);
    if (n < 2) {                                           // one part is its own sum
        if (n == 1 && scribe) sum[(size_t)slot * p.H + h] = dec[(size_t)slot * p.H + h];
        return;
    }
    const long step = forwards ? p.H : -(long)p.H;
    const size_t at = (size_t)(forwards ? slot : slot + n - 1) * p.H + h;
    const auto load = [&](int i) {
        return *reinterpret_cast<const f32x4 *>(part + (at + (long)min(i, n - 1) * step) * state + e);
    };
    // eight parts in flight; what is read again behind the last part is not used
    f32x4 S = {0.f, 0.f, 0.f, 0.f}, y[4] = {load(0), load(1), load(2), load(3)};
    float d = 1.f;
    for (int i0 = 0; i0 < n; i0 += 4) {
        f32x4 z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = load(i0 + 4 + j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j < n) {
                const size_t to = at + (i0 + j) * step;
                const float f = dec[to];
                S = S * f + y[j];
                *reinterpret_cast<f32x4 *>(part + to * state + e) = S;
                d *= f;
                if (scribe) sum[to] = d;
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = z[j];
    }
}

// dV (waves 0-3) and dK (waves 4-7) of one segment for one value head, chunks
// backwards, from one staging of q, k, v and dO; and dg.  With the terms
//   y_t = q_t . (state part of dq_t)            (from WALK_DQ_DG)
//   z_s = k_s . (state part of dk_s)
//   x_ts = scale D_ts (q_t . k_s)(dO_t . v_s),  t > s
//   w = e^{G_end} <S, dS>                       (S enters, dS leaves the chunk)
//   dg_u = sum_{t >= u} y_t + sum_{s < u} z_s + sum_{s < u <= t} x_ts + w
// and each sum is formed from its own terms alone (a running sum of what enters and leaves it would leave the large
// terms' roundings in the small sums behind a strong decay): the pairs by tiles of 16 x 16, on the diagonal summed over
// t >= u in the products' registers, and elsewhere as prefix and suffix sums inside a tile of 16 tokens plus
// totals of whole tiles.  w follows from R = <state, its gradient> at the chunk's end:
// w = R - sum z, and R at the chunk's start is w + sum y, both in float64; R is formed anew
// from the state that WALK_DQ_DG left at every anchor.  R carries the float32 roundings of the terms that it has passed
// since then, whose magnitudes M adds up, and so does w.  Where the chunk forgets (e^{G_end} < 2^-24) and R - sum z is
// not above those roundings (2^-22 M, two bits above one of M), w is 0, so that they do not reach the tokens before.
// The decay alone does not say so: a state that is large next to what the chunk adds leaves a w above them.
// One workgroup fills a compute unit (96 KiB of LDS, 8 waves of up to 256 registers); it is bound by
// latency: the matrix cores are busy 22% of the time, and the waves wait for LDS, barriers and one another for 40% of theirs.
// T = 8192, H = 32, d = 128, bf16: 196 to 239 us with dg, of a call's 355 to 365 us, 150 to 199 us without (kernel
// traces; with dg 94 scalar registers are kept in lanes of a vector register, without it 5).
template <typename T, int DK, int DV> struct DkdvLds {
    static constexpr int C = chunk_of<T>, LK = ld_of<T>(DK), LV = ld_of<T>(DV), LP = ldp_of<T>;
    T q[C * LK], k[C * LK], v[C * LV], d_o[C * LV];
    T p[2][C * LP];           // decayed scores of dV and of dK
    Decay<C> decay[2];
    float z[NW][C];           // by wave: sums over its columns
    // x summed over the 16 s of a tile (for each t, by the tile's s), over its 16 t (for each s, by its t); 0 where no
    // tile is.  On the diagonal x_t holds the tile's sum over s < u <= t for each u, and x_s is 0.
    float x_t[C / 16][C], x_s[C / 16][C];
    double r[NW];             // by wave: <state, gradient> at an anchor
};

// The walk of one kind of waves; both kinds pass the same barriers.
template <typename T, int DK, int DV, bool DG, bool KEYS>
__device__ __forceinline__ void dkdv_walk(const LinearBwdParams &b, DkdvLds<T, DK, DV> &s, const Piece &w, int id, int h)
{
    const LinearChunkParams &p = b.c;
    using L = DkdvLds<T, DK, DV>;
    constexpr int THREADS = 128 * NW;
    using GV = Group<T, DK, DV, true>;    // rows k, sources q, values dO, state dS
    using GK = Group<T, DV, DK, true>;    // rows v, sources dO, values q, state dS^T
    using G = typename std::conditional<KEYS, GK, GV>::type;
    constexpr int C = G::C, NT = G::NT;
    const int t = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(t >> 6) & (NW - 1);
    const bool scribe = !KEYS && wv == NW - 1;                 // forms the decays and dg: the wave with the fewest scores
    const int first = w.part * p.seg, toks = min(p.seg, w.len - first);
    const int nc = (max(toks, 0) + C - 1) / C;
    const int row0 = w.begin + first;
    const int hk = h / p.group, Hk = p.H / p.group;
    const size_t sk = (size_t)Hk * DK, sv = (size_t)p.H * DV;
    const size_t pair = (size_t)w.seq * p.H + h, part_size = (size_t)DK * DV;

    G grp;
    grp.clear();
    if (b.dhT) grp.template add<KEYS>(b.dhT + pair * part_size, 0.f, wv);
    for (int i = p.summed ? min(w.part + 1, w.parts - 1) : w.parts - 1; i > w.part; --i) {
        if (w.slot + i - 1 >= p.n_part) continue;
        const size_t at = (size_t)(w.slot + i - 1) * p.H + h;
        if constexpr (KEYS)
            grp.template add<true>(p.part_tr + at * part_size, p.dec[at], wv);
        else
            grp.add_part(p.part + at * part_size, p.dec[at], wv);
    }
    Stage<T, DK, THREADS> rq, rk;
    Stage<T, DV, THREADS> rv, ro;
    G::clear_scores(s.p[KEYS], wv);
    if (DG && KEYS)
        for (int e = t - 64 * NW; e < NT * C; e += 64 * NW) s.x_t[e / C][e % C] = s.x_s[e / C][e % C] = 0.f;
    float rg = 0.f, ry = 0.f;
    size_t at_k = (size_t)(row0 + max(nc - 1, 0) * C) * sk + (size_t)hk * DK;   // the next chunk's rows
    size_t at_v = (size_t)(row0 + max(nc - 1, 0) * C) * sv + (size_t)h * DV;
    auto fetch = [&](int c) {
        const int row = row0 + c * C, n = min(C, toks - c * C);
        rq.load((const T *)p.q + at_k, sk, n, t);
        rk.load((const T *)p.k + at_k, sk, n, t);
        rv.load((const T *)p.v + at_v, sv, n, t);
        ro.load((const T *)b.d_o + at_v, sv, n, t);
        at_k -= C * sk;
        at_v -= C * sv;
        if (scribe) {
            if (DG) ry = lane_id() < n ? p.y[(size_t)(row + lane_id()) * p.H + h] : 0.f;
        }
    };
    auto decays_of = [&](int c) { return fetch_decay(p, row0 + c * C, h, min(C, toks - c * C)); };
    if (nc > 0) {
        fetch(nc - 1);
        if (scribe) {
            make_decay<C, true>(&s.decay[0], decays_of(nc - 1), p.scale);
            if (nc > 1) rg = decays_of(nc - 2);
        }
    }
    double R = 0.0, sum_dg = 0.0;
    float M = 0.f;
    for (int i = 0; i < nc; ++i) {
        const int c = nc - 1 - i, n = min(C, toks - c * C), row = row0 + c * C;
        const int pos = first + c * C + n;
        const Decay<C> &d = s.decay[i & 1];
        const long anchor = DG ? anchor_at(p, w, pos) : -1;
        lds_barrier();                                         // the last chunk has been read
        rq.store(s.q, t);
        rk.store(s.k, t);
        rv.store(s.v, t);
        ro.store(s.d_o, t);
        const float y = ry;
        lds_barrier();
        if constexpr (DG && KEYS)                              // before the next loads: they would be waited for with it
            if (anchor >= 0) {
                const double r = grp.template dot<true>(p.anchors + ((size_t)anchor * p.H + h) * part_size, wv);
                if (lane_id() == 0) s.r[wv] = r;
            }
        if (i + 1 < nc) fetch(c - 1);
        f32x4 O[NT][G::NCT];
        if constexpr (!KEYS) {
            if constexpr (DG) {
                // the pair terms x of each tile too, summed along both axes
                const int l = lane_id(), x = l & 15, g = l >> 4;
                G::for_tiles(wv, [&](int rt, int st) {
                    const f32x4 a = G::decayed(G::scores(s.k, s.q, rt, st), d, p.scale, rt, st);
                    const f32x4 dov = GK::scores(s.v, s.d_o, rt, st);
                    G::put_scores(s.p[0], a, rt, st);
                    f32x4 xs = a * dov;
                    if (rt == st) {                            // a lane's s is x, its t are 4 g .. + 3
                        xs[2] += xs[3];
                        xs[1] += xs[2];
                        xs[0] += xs[1];
                        const float pair = __shfl_xor(xs[0], 16), half = __shfl_xor(xs[0] + pair, 32);
                        const float later = ((g & 1) == 0 ? pair : 0.f) + (g < 2 ? half : 0.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) xs[e] = x < 4 * g + e ? xs[e] + later : 0.f;
                    } else {
                        float over = (xs[0] + xs[1]) + (xs[2] + xs[3]);
                        over += __shfl_xor(over, 16);
                        over += __shfl_xor(over, 32);
                        if (g == 0) s.x_s[st][16 * rt + x] = over;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) xs[e] = row_total(xs[e]);
                    if (x == 0) *reinterpret_cast<f32x4 *>(&s.x_t[rt][16 * st + 4 * g]) = xs;
                });
            } else {
                G::make_scores(s.p[0], s.k, s.q, d, p.scale, wv);
            }
            grp.template inter<1>(O, s.k, d);
            if (scribe && i + 1 < nc) {
                const float x = rg;
                if (i + 2 < nc) rg = decays_of(c - 2);
                make_decay<C, true>(&s.decay[(i + 1) & 1], x, p.scale);
            }
        } else {
            G::make_scores(s.p[1], s.v, s.d_o, d, p.scale, wv);
            if constexpr (DG) {
                const int x = lane_id() & 15;
                grp.template inter<split_of<T>>(O, s.v, d);
                G::row_dots(s.z[wv], [&](int it, int ct) {
                    return *reinterpret_cast<const quad_t<T> *>(s.k + (16 * it + x) * L::LK + G::first_col(wv) + 4 * ct);
                }, O);
            } else {
                grp.template inter<1>(O, s.v, d);
            }
        }
        lds_barrier();                                         // scores and sums are whole
        if constexpr (!KEYS) {
            G::intra(O, s.p[0], s.d_o, wv);
            G::store((T *)b.dv + ((size_t)row * p.H + h) * DV, sv, n, O, wv);
            grp.update(s.q, s.d_o, d, wv);
            if (DG && scribe) {
                const int u = lane_id(), tile = u >> 4;
                float z = 0.f, yu = 0.f, own = 0.f, from = 0.f, to = 0.f, over[NT] = {};
                if (u < C) {
#pragma unroll
                    for (int j = 0; j < NW; ++j) z += s.z[j][u];
                    yu = y;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float x = s.x_t[j][u];           // u as t, s in tile j
                        own = tile == j ? x : own;
                        if (j > 0 && j + 1 < NT) over[j] = tile > j ? to : 0.f;
                        to += tile > j ? x : 0.f;
                        from += s.x_s[j][u];                   // u as s, t in tile j
                    }
                }
                if (anchor >= 0) {
                    R = 0.0;
#pragma unroll
                    for (int j = 0; j < NW; ++j) R += s.r[j];
                    M = fabsf((float)R);
                }
                // inside the tile; then the other tiles' y behind it, z before it and pairs over it
                float dg = (own + row_from(yu + to)) + row_before(z + from);
                const float yt = row_total(yu), zt = row_total(z);
                double ys = 0.0, zs = 0.0;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float yj = lane_value(yt, 16 * j), zj = lane_value(zt, 16 * j);
                    ys += (double)yj;
                    zs += (double)zj;
                    dg += (tile < j ? yj : 0.f) + (tile > j ? zj : 0.f);
                }
#pragma unroll
                for (int j = 1; j + 1 < NT; ++j) {
                    const float pairs = wave_sum(over[j]);
                    dg += tile == j ? pairs : 0.f;
                }
                double wt = R - zs;
                M += wave_sum(fabsf(z));
                if (d.total == 0.f || (d.total < 0x1p-24f && fabs(wt) <= 0x1p-22 * (double)M)) wt = M = 0.f;
                if (c == 0 && w.part == 0 && !p.h0) wt = 0.0;  // no state enters
                R = wt + ys;
                M += wave_sum(fabsf(yu));
                dg += (float)wt;
                if (u < n) {
                    if (p.g_per_head) sum_dg += dg; else b.dg[(size_t)(row + u) * p.H + h] = dg;
                }
            }
        } else {
            G::intra(O, s.p[1], s.q, wv);
            if (p.wide)
                G::store((float *)b.dk + ((size_t)row * p.H + h) * DK, (size_t)p.H * DK, n, O, wv);
            else
                G::store((T *)b.dk + ((size_t)row * Hk + hk) * DK, sk, n, O, wv);
            grp.update(s.d_o, s.q, d, wv);
        }
    }
    if constexpr (!KEYS) {
        if (w.part == 0 && b.dh0)
            grp.template put<false>(deferred(p, w, 0) ? p.part + ((size_t)w.slot * p.H + h) * part_size
                                                      : b.dh0 + pair * part_size, wv);
        if (DG && p.g_per_head && scribe) {
            sum_dg = wave_total(sum_dg);
            if (lane_id() == 0) b.dg_part[(size_t)id * p.H + h] = sum_dg;
        }
    }
}

template <typename T, int DK, int DV, bool DG>
__global__ __launch_bounds__(128 * NW, 2) void linear_dkdv_kernel(const LinearBwdParams b)
{
    extern __shared__ __align__(16) char smem[];
    DkdvLds<T, DK, DV> &s = *reinterpret_cast<DkdvLds<T, DK, DV> *>(smem);
    const int h = (int)(blockIdx.x % (unsigned)b.c.H), id = (int)(blockIdx.x / (unsigned)b.c.H);
    Piece w;
    if (!find_piece(b.c, id, w)) return;
    if (__builtin_amdgcn_readfirstlane(threadIdx.x) >= 64 * NW)
        dkdv_walk<T, DK, DV, DG, true>(b, s, w, id, h);
    else
        dkdv_walk<T, DK, DV, DG, false>(b, s, w, id, h);
}

// dg of constant decays: the segments' sums in order.  One wave per head.
__global__ __launch_bounds__(64) void linear_dg_heads_kernel(const LinearBwdParams b, int cap)
{
    const LinearChunkParams &p = b.c;
    const int h = (int)blockIdx.x;
    Piece w;
    int lo = 0, hi = cap;                 // segments there are: the first id that is none
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (find_piece(p, mid, w)) lo = mid + 1; else hi = mid;
    }
    double s = 0.0;
    for (int i = lane_id(); i < lo; i += 64) s += b.dg_part[(size_t)i * p.H + h];
    s = wave_total(s);
    if (lane_id() == 0) b.dg[h] = (float)s;
}

// Gradients of shared query / key heads: the sum over their value heads, for the rows that sequences cover.
template <typename T>
__global__ __launch_bounds__(256) void linear_share_kernel(const LinearChunkParams p, const float *dq, const float *dk, T *oq, T *ok, int DK)
{
    int lo = 0, hi = p.rows;
    if (p.cu) {
        lo = min(max(p.cu[0], 0), p.T);
        hi = min(max(p.cu[p.N], lo), p.T);
    }
    const int Hk = p.H / p.group, per = DK / 4;
    const size_t n = (size_t)(hi - lo) * Hk * per;
    const float *src = blockIdx.y ? dk : dq;
    T *dst = blockIdx.y ? ok : oq;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        const size_t head = (size_t)lo * Hk + i / per;         // (row, query / key head)
        const float *s = src + head * p.group * DK + (i % per) * 4;
        f32x4 a = *reinterpret_cast<const f32x4 *>(s);
        for (int j = 1; j < p.group; ++j) a += *reinterpret_cast<const f32x4 *>(s + (size_t)j * DK);
        *reinterpret_cast<quad_t<T> *>(dst + head * DK + (i % per) * 4) = make_quad<T>(a);
    }
}

// ---- launches ----------------------------------------------------------------------------------------------------------

template <typename T, int DK, int DV> static hipError_t fwd_t(const LinearChunkParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((size_t)p.n_seg * p.H)), block(64 * NW);
    static_assert(64 * NW <= LINEAR_FWD_THREADS && 128 * NW <= LINEAR_BWD_THREADS, "grids are checked for these");
    hipError_t e = launch_table(p, stream);
    if (e != hipSuccess) return e;
    if (p.part) {
        hipLaunchKernelGGL((linear_walk_kernel<T, DK, DV, WALK_STATE>), grid, block, 0, stream, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((linear_walk_kernel<T, DK, DV, WALK_OUT>), grid, block, 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess || !p.defer) return e;
    hipLaunchKernelGGL(linear_deferred_kernel, grid, block, 0, stream, p, p.hT, 0, DK * DV);
    return hipGetLastError();
}

template <typename T, int DK, int DV> static hipError_t bwd_t(const LinearBwdParams &b, hipStream_t stream)
{
    const LinearChunkParams &c = b.c;
    const dim3 grid((unsigned)((size_t)c.n_seg * c.H)), block(64 * NW);
    hipError_t e = launch_table(c, stream);
    if (e != hipSuccess) return e;
    LinearChunkParams dq = c;
    if (c.part) {
        LinearChunkParams s = c;
        s.part = b.part_fwd; s.dec = b.dec_fwd;
        s.k = c.v; s.v = c.k;
        hipLaunchKernelGGL((linear_walk_kernel<T, DV, DK, WALK_STATE_DQ>), grid, block, 0, stream, s);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        s = c;
        s.k = c.q; s.v = b.d_o;
        hipLaunchKernelGGL((linear_walk_kernel<T, DK, DV, WALK_STATE_REV>), grid, block, 0, stream, s);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        dq.part = b.part_fwd; dq.dec = b.dec_fwd;
        if (c.summed) {
            hipLaunchKernelGGL(linear_scan_kernel, dim3(c.N * c.H, 3, DK * DV / 1024), dim3(256), 0, stream, b, DK * DV);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            dq.dec = b.sum_fwd;
        }
    }
    dq.q = b.d_o; dq.k = c.v; dq.v = c.k; dq.q_rows = c.q; dq.o = b.dq;
    if (b.dg)
        hipLaunchKernelGGL((linear_walk_kernel<T, DV, DK, WALK_DQ_DG>), grid, block, 0, stream, dq);
    else
        hipLaunchKernelGGL((linear_walk_kernel<T, DV, DK, WALK_DQ>), grid, block, 0, stream, dq);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    constexpr size_t lds = sizeof(DkdvLds<T, DK, DV>);
    static_assert(lds <= 160 * 1024, "one compute unit's LDS");
    const auto kernel = b.dg ? linear_dkdv_kernel<T, DK, DV, true> : linear_dkdv_kernel<T, DK, DV, false>;
    // above 64 KiB a kernel asks for its dynamic LDS; per device, so with every launch
    e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    LinearBwdParams kv = b;
    if (c.summed) kv.c.dec = b.sum_rev;
    hipLaunchKernelGGL(kernel, grid, dim3(128 * NW), lds, stream, kv);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (c.defer) {
        hipLaunchKernelGGL(linear_deferred_kernel, grid, block, 0, stream, c, b.dh0, 1, DK * DV);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (b.dg && c.g_per_head) {
        hipLaunchKernelGGL(linear_dg_heads_kernel, dim3((unsigned)c.H), dim3(64), 0, stream, b, c.n_seg);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (c.wide) {
        hipLaunchKernelGGL((linear_share_kernel<T>), dim3(2048, 2), dim3(256), 0, stream, c, (const float *)b.dq,
                           (const float *)b.dk, (T *)b.dq_out, (T *)b.dk_out, DK);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

#define KDA_LINEAR_DISPATCH(FN, ARG)                                              \
    if (dtype_bf16) {                                                             \
        if (Dk == 64 && Dv == 64) return FN<bf16, 64, 64>(ARG, stream);           \
        if (Dk == 64 && Dv == 128) return FN<bf16, 64, 128>(ARG, stream);         \
        if (Dk == 128 && Dv == 64) return FN<bf16, 128, 64>(ARG, stream);         \
        if (Dk == 128 && Dv == 128) return FN<bf16, 128, 128>(ARG, stream);       \
    } else {                                                                      \
        if (Dk == 64 && Dv == 64) return FN<float, 64, 64>(ARG, stream);          \
        if (Dk == 64 && Dv == 128) return FN<float, 64, 128>(ARG, stream);        \
        if (Dk == 128 && Dv == 64) return FN<float, 128, 64>(ARG, stream);        \
        if (Dk == 128 && Dv == 128) return FN<float, 128, 128>(ARG, stream);      \
    }                                                                             \
    return hipErrorInvalidValue;

hipError_t launch_linear_fwd(int dtype_bf16, int Dk, int Dv, const LinearChunkParams &p, hipStream_t stream)
{
    KDA_LINEAR_DISPATCH(fwd_t, p)
}

hipError_t launch_linear_bwd(int dtype_bf16, int Dk, int Dv, const LinearBwdParams &p, hipStream_t stream)
{
    KDA_LINEAR_DISPATCH(bwd_t, p)
}

}  // namespace kda

// kda_block_dev.h -- device-side building blocks of the gated scan, the norms
// around a block and 8-bit activations: eight consecutive channels a lane.
#pragma once

#include "kda_block.h"
#include "kda_common.h"

namespace kda {

constexpr int LANE_CH = 8;            // channels a lane holds: 16 bytes of bf16, one lane's share of a group of 128
constexpr float LOG2E = 1.44269504088896340736f;

// Global memory takes 16-byte accesses at any element address, so rows of odd
// length need no path of their own but for the last, shorter group of 8.
typedef __bf16 bf16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef int8_t i8x8_any __attribute__((ext_vector_type(8), aligned(1)));

// Channels [c, c + n) of a row, n in 0..8 (the rest 0).
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    bf16x8 v;
    __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
    __device__ __forceinline__ void load(const bf16 *p, int n)
    {
        if (n == 8) {
            v = *reinterpret_cast<const bf16x8_any *>(p);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : (bf16)0.f;
    }
    __device__ static __forceinline__ void store(bf16 *p, int n, const float *x)
    {
        if (n == 8) {
            bf16x8 f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (bf16)x[i];
            *reinterpret_cast<bf16x8_any *>(p) = f;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (bf16)x[i];
    }
};
template <> struct Raw8<float> {
    f32x4 a, b;
    __device__ __forceinline__ float operator[](int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
    __device__ __forceinline__ void load(const float *p, int n)
    {
        if (n == 8) {
            a = *reinterpret_cast<const f32x4_any *>(p);
            b = *reinterpret_cast<const f32x4_any *>(p + 4);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = i < n ? p[i] : 0.f;
            b[i] = i + 4 < n ? p[i + 4] : 0.f;
        }
    }
    __device__ static __forceinline__ void store(float *p, int n, const float *x)
    {
        if (n == 8) {
            const f32x4 lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
            *reinterpret_cast<f32x4_any *>(p) = lo;
            *reinterpret_cast<f32x4_any *>(p + 4) = hi;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = x[i];
    }
};

// The same for four channels.
typedef __bf16 bf16x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <typename T> struct Raw4;
template <> struct Raw4<bf16> {
    bf16x4 v;
    __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
    __device__ __forceinline__ void load(const bf16 *p, int n)
    {
        if (n == 4) {
            v = *reinterpret_cast<const bf16x4_any *>(p);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : (bf16)0.f;
    }
    __device__ static __forceinline__ void store(bf16 *p, int n, const float *x)
    {
        if (n == 4) {
            const bf16x4 f = {(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
            *reinterpret_cast<bf16x4_any *>(p) = f;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = (bf16)x[i];
    }
};
template <> struct Raw4<float> {
    f32x4 v;
    __device__ __forceinline__ float operator[](int i) const { return v[i]; }
    __device__ __forceinline__ void load(const float *p, int n)
    {
        if (n == 4) {
            v = *reinterpret_cast<const f32x4_any *>(p);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
    }
    __device__ static __forceinline__ void store(float *p, int n, const float *x)
    {
        if (n == 4) {
            const f32x4 f = {x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4_any *>(p) = f;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = x[i];
    }
};
__device__ __forceinline__ void load_f4(const float *p, int n, float *x)
{
    Raw4<float> raw;
    raw.load(p, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = raw[i];
}

__device__ __forceinline__ int act_groups(int C) { return (C + ACT_GROUP - 1) / ACT_GROUP; }

// Channels [c, c + n) of a row of codes, as values; scales: the row's.
__device__ __forceinline__ void load_codes(const int8_t *row, const float *scales, int c, int n, float *x)
{
    const float s = n > 0 ? scales[c / ACT_GROUP] : 0.f;
    if (n == 8) {
        const i8x8_any q = *reinterpret_cast<const i8x8_any *>(row + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)q[i] * s;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? (float)row[c + i] * s : 0.f;
}

__device__ __forceinline__ void load_f8(const float *p, int n, float *x)
{
    Raw8<float> raw;
    raw.load(p, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = raw[i];
}

// The largest of |x| over the 128 / CH lanes that hold a group (a DPP row, or two), as bits: integers order
// non-negative floats, and infinities and NaN above them.  All 64 lanes are active.
template <int CTRL> __device__ __forceinline__ uint32_t dpp_umax(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return o > v ? o : v;
}
template <int CH> __device__ __forceinline__ uint32_t group_amax(const float *x)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    m = dpp_umax<0xB1>(m);   // quad_perm [1, 0, 3, 2]
    m = dpp_umax<0x4E>(m);   // quad_perm [2, 3, 0, 1]
    m = dpp_umax<0x141>(m);  // row_half_mirror
    m = dpp_umax<0x140>(m);  // row_mirror
    if (CH == 4) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_ds_swizzle((int)m, 0x401F);  // lane ^ 16
        m = o > m ? o : m;
    }
    return m;
}

// Packs the lane's channels [c, c + n) of row r; x holds 0 from n on.  A group
// with an infinity or a NaN stands for NaN throughout (its scale is NaN); one whose largest value
// is below 2^-118 (127 over it would overflow) stands for zeros.
template <int CH> __device__ __forceinline__ void store_codes(const PackedOut &out, size_t r, int C, int c, int n, const float *x)
{
    typedef int8_t codes_any __attribute__((ext_vector_type(CH), aligned(1)));
    const uint32_t bits = group_amax<CH>(x);
    const float amax = __builtin_bit_cast(float, bits);
    const bool finite = bits < 0x7f800000u, some = bits >= 0x04800000u;
    const float inv = finite && some ? 127.0f / amax : 0.f;
    if (n == 0) return;
    if (c % ACT_GROUP == 0)
        out.scales[r * act_groups(C) + c / ACT_GROUP] =
            !finite ? __builtin_bit_cast(float, 0x7fc00000u) : some ? amax * (1.0f / 127.0f) : 0.f;
    codes_any q;
#pragma unroll
    for (int i = 0; i < CH; ++i) q[i] = finite ? (int8_t)(int)__builtin_rintf(x[i] * inv) : (int8_t)0;
    int8_t *p = out.codes + r * C + c;
    if (n == CH) {
        *reinterpret_cast<codes_any *>(p) = q;
        return;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
        if (i < n) p[i] = q[i];
}

// 1 / sqrt(mean of squares + eps): as rsq_norm, but a NaN stays one.
__device__ __forceinline__ float rstd_of(float x)
{
    return __builtin_amdgcn_rsqf(x < 1.17549435e-38f ? 1.17549435e-38f : x);
}

struct Sigmoid {
    float s, r;                       // Sigmoid(x) and 1 - Sigmoid(x), each to a few units in its own last place
};
__device__ __forceinline__ Sigmoid sigmoid2(float x)
{
    // below 2^-120 it counts as 0, so that neither part overflows
    const float y = x * -LOG2E;
    const bool shut = y > 120.f;
    const float e = __builtin_amdgcn_exp2f(shut ? 120.f : y);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    return {shut ? 0.f : s, e * s};
}

// The sum over `rows` rows of column blockIdx.x * 16 + thread % 16 of a matrix of C columns, on threads 0 .. 15 of 16 SLICES: in
// float64, in a fixed order.
template <int SLICES> __device__ __forceinline__ double column_sum(const float *part, int rows, int C, double (*s)[16])
{
    const int l = threadIdx.x & 15, slice = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
    double sum = 0.0;
    for (int i = slice; i < rows; i += 8 * SLICES) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = c < C && i + SLICES * u < rows ? part[(size_t)(i + SLICES * u) * C + c] : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += v[u];
    }
    s[slice][l] = sum;
    __syncthreads();
    if (slice > 0) return 0.0;
    for (int k = 1; k < SLICES; ++k) sum += s[k][l];
    return sum;
}

// A decay e^x (x <= 0, and -0 for 0) kept as one number w: e^x - 1, its sign set, where x > -0.1 (to its own last
// place: the cubic is within 1.3e-8 < 2^-25 of (e^x - 1) / x there, fitted to the least largest error); else e^x, its sign clear.
// A state that fades over 10^4 tokens would carry 10^4 times the rounding of e^x itself.
struct Decay {
    float w;
    bool near;
};
constexpr float NEAR = -0.1f, NEAR1 = 0.4999980032444f, NEAR2 = 0.16656582057476044f, NEAR3 = 0.040039222687482834f;
__device__ __forceinline__ Decay decay_of(float x)
{
    const float m = x * __builtin_fmaf(x, __builtin_fmaf(x, __builtin_fmaf(x, NEAR3, NEAR2), NEAR1), 1.f);
    const bool near = x > NEAR;
    return {near ? m : __builtin_amdgcn_exp2f(x * LOG2E), near};
}
// A log-decay above 0 counts as 0; NaN passes.
__device__ __forceinline__ float not_above_0(float g) { return g >= 0.f ? -0.f : g; }
__device__ __forceinline__ Decay decay_held(float w) { return {w, __builtin_bit_cast(int, w) < 0}; }
// e^x h + b.  An infinite h may give NaN (inf - 0.05 inf).
__device__ __forceinline__ float decay_apply(Decay d, float h, float b) { return (d.near ? h : 0.f) + __builtin_fmaf(d.w, h, b); }
__device__ __forceinline__ float decay_times(Decay d, float h) { return __builtin_fmaf(d.w, h, d.near ? h : 0.f); }
// The product of two decays.
__device__ __forceinline__ Decay decay_product(Decay a, Decay b)
{
    const float t = __builtin_fmaf(a.w, b.w, (b.near ? a.w : 0.f) + (a.near ? b.w : 0.f));
    // near 1 it stays e^x - 1 as long as that keeps its last place
    const bool near = a.near && b.near;
    return near && t < -0.5f ? Decay{1.f + t, false} : Decay{near ? -__builtin_fabsf(t) : t, near};  // (-0 for 1)
}
// What a token's value is multiplied by: 1 - e^x with complement, else 1.
__device__ __forceinline__ float share_of(Decay d, float x, bool complement)
{
    return complement ? __builtin_fmaf(-d.w, x, d.near ? 0.f : x) : x;
}
// One token: e^x h + v, or with complement e^x h + (1 - e^x) v = v + e^x (h - v).
__device__ __forceinline__ float decay_step(Decay d, float h, float v, bool complement)
{
    return complement ? __builtin_fmaf(d.w, h - v, d.near ? h : v) : decay_apply(d, h, v);
}

}  // namespace kda

// kda_block_norm.hip -- what stands between two blocks of a model:
//   u = w_post y / rms(y),  x' = x + s Sigmoid(gate) u,  n = w_pre x' / rms(x'),
// and its gradients.
#include "kda_block_dev.h"

namespace kda {

// Sums of K values over the NW waves that hold a row, on every lane.  The waves' sums pass through LDS, where each
// 16 lanes read one a lane and add them up among themselves; two buffers in turn, so that one barrier a sum is enough.
template <int NW, int K> struct RowSum {
    float (*lds)[K][NW];
    int turn;
    __device__ __forceinline__ void operator()(float *v)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
        if constexpr (NW > 1) {
            const int wave = threadIdx.x / 64 % NW;        // of the row
            if (lane_id() == 0)
#pragma unroll
                for (int k = 0; k < K; ++k) lds[turn][k][wave] = v[k];
            lds_barrier();
            const int w = threadIdx.x % 16;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float x = lds[turn][k][w % NW];
                x = w < NW ? x : 0.f;
                x = dpp_add<0xB1, 0xF>(x);                 // quad_perm [1, 0, 3, 2]
                x = dpp_add<0x4E, 0xF>(x);                 // quad_perm [2, 3, 0, 1]
                x = dpp_add<0x141, 0xF>(x);                // row_half_mirror
                v[k] = dpp_add<0x140, 0xF>(x);             // row_mirror
            }
            turn ^= 1;
        }
    }
};

// Six such sums at once: lanes trade values while they add (8, 4, 2 of them a lane), so that a wave needs 30 instructions
// instead of 42 and the waves' sums 14 instead of 30; uniform results.
__device__ __forceinline__ float rows_add(float v)                                    // over the four rows of 16 lanes
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    auto a = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t c = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]));
    a = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}
template <int NW> struct RowSum6 {
    float (*lds)[NW][8];
    int turn;
    __device__ __forceinline__ void operator()(float *v)
    {
        const int lane = lane_id();
        const bool odd = lane & 1, high = lane & 2;
        float a[4], b[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {                       // value k or k + 4
            const float other = k < 2 ? v[k + 4] : 0.f;
            a[k] = (odd ? other : v[k]) + dpp_move<0xB1>(odd ? v[k] : other);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            b[k] = (high ? a[k + 2] : a[k]) + dpp_move<0x4E>(high ? a[k] : a[k + 2]);
            b[k] = dpp_add<0x128, 0xF>(b[k]);               // row_ror:8
            b[k] = dpp_add<0x124, 0xF>(b[k]);               // row_ror:4
            b[k] = rows_add(b[k]);
        }
        // lane l now has values 4 (l & 1) + (l & 2) and the next one
        if constexpr (NW == 1) {
#pragma unroll
            for (int k = 0; k < 6; ++k) v[k] = read_lane(b[k % 2], k / 4 + (k & 2));
        } else {
            const int wave = threadIdx.x / 64 % NW;
            if (lane < 4) {
                lds[turn][wave][4 * (lane & 1) + (lane & 2)] = b[0];
                lds[turn][wave][4 * (lane & 1) + (lane & 2) + 1] = b[1];
            }
            lds_barrier();
            float x = lds[turn][lane / 8 % NW][lane % 8];
            if (NW == 16) x += lds[turn][(lane / 8 + 8) % NW][lane % 8];
            if (NW < 8) x = lane / 8 < NW ? x : 0.f;
            x = rows_add(dpp_add<0x128, 0xF>(x));
#pragma unroll
            for (int k = 0; k < 6; ++k) v[k] = read_lane(x, k);
            turn ^= 1;
        }
    }
    template <int CTRL> __device__ static __forceinline__ float dpp_move(float v)
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
    }
    __device__ static __forceinline__ float read_lane(float v, int l)
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    }
};

template <int V, typename A, typename B> struct Pick { typedef A type; };
template <typename A, typename B> struct Pick<8, A, B> { typedef B type; };

// A uniform address and a lane's 32-bit offset.
template <typename T> __device__ __forceinline__ T *at_byte(T *p, unsigned bytes)
{
    return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + bytes);
}

// V (4 or 8) channels of a row as they are stored: elements, or codes with their scale.
template <typename T, int V> struct HeldV {
    static constexpr int WORDS = V * sizeof(T) / 4;
    typedef typename Pick<V, Raw4<T>, Raw8<T>>::type Raw;
    uint32_t v[WORDS];
    // r is uniform
    __device__ __forceinline__ void load(const Rows &m, size_t r, int D, unsigned c, int n)
    {
        if (m.scales) {
            const int8_t *at = (const int8_t *)m.p + r * m.stride + c;
            if (n == V) {
                typedef uint32_t codes_any __attribute__((ext_vector_type(V / 4), aligned(1)));
                const codes_any q = *reinterpret_cast<const codes_any *>(at);
#pragma unroll
                for (int k = 0; k < V / 4; ++k) v[k] = q[k];
            } else {
                v[0] = v[V / 4 - 1] = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < n) v[i / 4] |= (uint32_t)(uint8_t)at[i] << (8 * (i % 4));
            }
            v[V / 4] = n > 0 ? __builtin_bit_cast(uint32_t, *at_byte(m.scales + r * act_groups(D), c / ACT_GROUP * 4)) : 0;
            return;
        }
        Raw raw;
        raw.load(at_byte((const T *)m.p + r * m.stride, c * sizeof(T)), n);
        __builtin_memcpy(v, &raw, sizeof(raw));
    }
    // channels [4 k, 4 k + 4)
    __device__ __forceinline__ void get(bool packed, int k, float *x) const
    {
        if (packed) {
            const float s = __builtin_bit_cast(float, v[V / 4]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(v[k] >> (8 * i)) * s;
            return;
        }
        Raw raw;
        __builtin_memcpy(&raw, v, sizeof(raw));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = raw[4 * k + i];
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void hold()                 // what is made from these words is not kept
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(v[i]));
    }
};

// A weight's channels of a lane, `otherwise` where there is no weight.
__device__ __forceinline__ void load_weight(const float *w, int c, int n, float otherwise, float *x)
{
    if (w) {
        load_f8(w + c, n, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = otherwise;
}

// Bound by memory (10 bytes an element in bf16, 13 to 16 backwards).  NW waves hold a row, 8 NCH channels a lane; a
// workgroup of ROWS such rows side by side goes through its rows with the weights in registers and the next rows'
// values on their way.

template <typename T, typename X, int NW, int ROWS, int NCH>
__global__ __launch_bounds__(64 * NW * ROWS, 4) void norm_fwd_kernel(const NormParams p)
{
    constexpr int NT = 64 * NW;                            // threads of a row
    __shared__ float s_sum[ROWS][2][1][NW];
    const int t = threadIdx.x % NT, side = threadIdx.x / NT;
    RowSum<NW, 1> sum = {s_sum[side], 0};
    constexpr bool HELD = NCH == 1;                        // weights and the next row stay in registers
    int cnt[NCH];
    float wpost[8], wres[8], wpre[8];
    const auto weights = [&](int j, bool after) {
        const int c = (j * NT + t) * LANE_CH;
        if (!after) {
            load_weight(p.post, c, cnt[j], 1.f, wpost);
            load_weight(p.res, c, cnt[j], 1.f, wres);
#pragma unroll
            for (int i = 0; i < 8; ++i) wres[i] *= p.scale;
        } else {
            load_weight(p.pre, c, cnt[j], 0.f, wpre);
        }
    };
#pragma unroll
    for (int j = 0; j < NCH; ++j) cnt[j] = max(0, min(LANE_CH, p.D - (j * NT + t) * LANE_CH));
    if (HELD) {
        weights(0, false);
        weights(0, true);
    }
    Raw8<X> xr[NCH];
    Raw8<T> yr[NCH], gr[NCH];
    const auto load = [&](int row) {
        const size_t r = min(row, p.R - 1);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = (j * NT + t) * LANE_CH;
            xr[j].load((const X *)p.x.p + r * p.D + c, cnt[j]);
            if (p.y.p) yr[j].load((const T *)p.y.p + r * p.y.stride + c, cnt[j]);
            if (p.gate.p) gr[j].load((const T *)p.gate.p + r * p.gate.stride + c, cnt[j]);
        }
    };
    const float inv_d = 1.f / (float)p.D;
    const int step = gridDim.x * ROWS;
    if (HELD) load(blockIdx.x * ROWS + side);
    // all sides stay while one has a row: sums are joined behind barriers
    for (int row0 = blockIdx.x * ROWS; row0 < p.R; row0 += step) {
        const int row = row0 + side;
        const bool in = row < p.R;
        const size_t r = min(row, p.R - 1);
        if (!HELD) load(row);
        float x[NCH][8], u[NCH][8], g[NCH][8];
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[j][i] = xr[j][i];
                if (p.y.p) u[j][i] = yr[j][i];
                if (p.gate.p) g[j][i] = gr[j][i];
            }
        if (HELD && row0 + step < p.R) load(row + step);
        if (p.y.p) {
            float rs = 1.f;
            if (p.post) {
#pragma unroll
                for (int j = 0; j < NCH; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss[0] += u[j][i] * u[j][i];
                sum(ss);
                rs = rstd_of(ss[0] * inv_d + p.eps);
            }
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH, n = in ? cnt[j] : 0;
                if (p.y8.codes) store_codes<LANE_CH>(p.y8, r, p.D, c, n, u[j]);
                if (p.gate8.codes) store_codes<LANE_CH>(p.gate8, r, p.D, c, n, g[j]);
                if (!HELD) weights(j, false);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v = wpost[i] * (u[j][i] * rs);
                    if (p.gate.p) v *= sigmoid2(g[j][i]).s;
                    x[j][i] = to_f<X>(from_f<X>(x[j][i] + wres[i] * v));
                }
                if (n > 0) Raw8<X>::store((X *)p.x_out + r * p.D + c, n, x[j]);
            }
        }
        if (p.x8.codes)
#pragma unroll
            for (int j = 0; j < NCH; ++j)
                store_codes<LANE_CH>(p.x8, r, p.D, (j * NT + t) * LANE_CH, in ? cnt[j] : 0, x[j]);
        if (p.pre) {
            ss[0] = 0.f;
#pragma unroll
            for (int j = 0; j < NCH; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] += x[j][i] * x[j][i];
            sum(ss);
            const float rs = rstd_of(ss[0] * inv_d + p.eps);
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH;
                if (!HELD) weights(j, true);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = wpre[i] * (x[j][i] * rs);
                if (in && cnt[j] > 0) Raw8<T>::store((T *)p.n + r * p.D + c, cnt[j], x[j]);
            }
        }
    }
}

// Four floats a lane for each of NQ pieces: in registers, or in LDS, where a lane reads and writes its own places only.
template <int NT, int NQ, bool LDS> struct Quads;
template <int NT, int NQ> struct Quads<NT, NQ, false> {
    f32x4 v[NQ];
    __device__ __forceinline__ void begin(float *) {}
    __device__ __forceinline__ f32x4 get(int j) const { return v[j]; }
    __device__ __forceinline__ void put(int j, f32x4 x) { v[j] = x; }
};
template <int NT, int NQ> struct Quads<NT, NQ, true> {
    f32x4 *at;
    __device__ __forceinline__ void begin(float *lds) { at = reinterpret_cast<f32x4 *>(lds) + threadIdx.x; }
    __device__ __forceinline__ f32x4 get(int j) const { return at[j * NT]; }
    __device__ __forceinline__ void put(int j, f32x4 x) { at[j * NT] = x; }
};

// Gradients.  One sum over the row is enough: with A = w_post Sigmoid(gate) s y,
//   sum of w_post du y = sum A dx + rx sum A w_pre dn - rx^2 mx sum A x,
// so a row has one barrier between its two looks at the values (two: 160 us for 8192 x 4096 from 8 bits).  NW waves hold a row,
// NQ times 4 channels a lane.  With 4 (up to 4096 channels) the weights, their sums, a row and the next one as it is stored fit
// 128 registers, so that 16 waves a unit hide the sum (8 channels a lane and 8 waves: 143 us).  With 8 the weights lie in LDS, with 16 two of
// the sums do and the weights are read again for every row; either unpacks the row's values a second time for the second look.
template <typename T, typename X, int NW, int ROWS, int NQ>
__global__ __launch_bounds__(64 * NW * ROWS, 4) void norm_bwd_kernel(const NormParams p)
{
    constexpr int NT = 64 * NW, V = NQ == 1 ? 4 : 8, NV = 4 * NQ / V;
    constexpr bool KEEP = NQ == 1;                         // numbers stay from look to look, the next row is on its way
    extern __shared__ __align__(16) float s_mem[];         // NQ 2: weights [3][2][NT][4]; 4: sums [2][4][NT][4]; at the end [ROWS - 1][3][NT][4]
    __shared__ float s_sum[ROWS][2][NW][8];
    const int t = threadIdx.x % NT, side = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    RowSum6<NW> total = {s_sum[side], 0};
    const bool block = p.y.p, pre = p.pre && p.d_n, gated = p.gate.p;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // With D a multiple of V a lane has V channels or none, and asks nothing more; else the last one goes by elements.
    const bool whole = p.D % V == 0;
    int cnt[NV];
#pragma unroll
    for (int g = 0; g < NV; ++g) cnt[g] = max(0, min(V, p.D - (g * NT + t) * V));
    const auto channel = [&](int j) { return (unsigned)((4 * j / V * NT + t) * V + 4 * j % V); };
    Quads<NT, NQ, NQ == 2> w_post, w_res, w_pre;
    Quads<NT, NQ, NQ == 4> a_post, a_res;
    Quads<NT, NQ, false> a_pre;
    a_post.begin(s_mem);
    a_res.begin(s_mem + 4 * NQ * NT);
    w_post.begin(s_mem);
    w_res.begin(s_mem + 4 * NQ * NT);
    w_pre.begin(s_mem + 8 * NQ * NT);
    const auto weights = [&](int j, f32x4 &post, f32x4 &res, f32x4 &pre_) {
        const unsigned c = channel(j);
        const int n = max(0, min(4, p.D - (int)c));
        float w[3][4] = {{1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}};
        if (p.post) load_f4(at_byte(p.post, 4 * c), n, w[0]);
        if (p.res) load_f4(at_byte(p.res, 4 * c), n, w[1]);
        if (p.pre) load_f4(at_byte(p.pre, 4 * c), n, w[2]);
        post = f32x4{w[0][0], w[0][1], w[0][2], w[0][3]};
        res = f32x4{w[1][0], w[1][1], w[1][2], w[1][3]} * p.scale;
        pre_ = f32x4{w[2][0], w[2][1], w[2][2], w[2][3]};
    };
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        if (NQ <= 2) {
            f32x4 a, b, c;
            weights(j, a, b, c);
            w_post.put(j, a);
            w_res.put(j, b);
            w_pre.put(j, c);
        }
        a_post.put(j, zero);
        a_res.put(j, zero);
        a_pre.put(j, zero);
    }
    const auto weight = [&](int j, f32x4 &post, f32x4 &res, f32x4 &pre_) {
        if (NQ > 2) {
            weights(j, post, res, pre_);
        } else {
            post = w_post.get(j);
            res = w_res.get(j);
            pre_ = w_pre.get(j);
        }
    };
    struct Values {
        HeldV<X, V> x[NV], dx[NV];
        HeldV<T, V> y[NV], gate[NV], dn[NV];
    };
    Values next;
    const Rows d_n = {p.d_n, nullptr, p.D}, d_x = {p.d_x, nullptr, p.D};
    const auto load_some = [&](size_t r, int g, int n) {
        const unsigned c = (g * NT + t) * V;
        if (block) next.y[g].load(p.y, r, p.D, c, n);
        if (pre) {
            next.x[g].load(p.x, r, p.D, c, n);
            next.dn[g].load(d_n, r, p.D, c, n);
        }
        if (p.d_x) next.dx[g].load(d_x, r, p.D, c, n);
        if (gated) next.gate[g].load(p.gate, r, p.D, c, n);
    };
    const auto load = [&](int row) {
        const size_t r = min(row, p.R - 1);
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            if (whole) {
                if (cnt[g] > 0) load_some(r, g, V);
            } else {
                load_some(r, g, cnt[g]);
            }
        }
    };
#pragma unroll
    for (int g = 0; g < NV; ++g) {                         // lanes without channels keep zeros
        next.y[g].clear();
        next.x[g].clear();
        next.dn[g].clear();
        next.dx[g].clear();
        next.gate[g].clear();
    }
    struct Floats {                                        // zeros (an open gate) where there is no such part
        float x[4], y[4], dx[4], dn[4];
        Sigmoid gate[4];
    };
    const float inv_d = 1.f / (float)p.D;
    const int step = p.parts * ROWS;
    if (KEEP) load(blockIdx.x * ROWS + side);
    for (int row0 = blockIdx.x * ROWS; row0 < p.R; row0 += step) {
        const int row = row0 + side;
        const bool in = ROWS == 1 || row < p.R;            // a side without a row adds zeros
        const size_t r = min(row, p.R - 1);
        if (!KEEP) load(row);
        Values now = next;
        if (KEEP && row0 + step < p.R) load(row + step);
        const auto floats = [&](int j, Floats &f) {
            const int g = 4 * j / V, k = j - g * V / 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f.x[i] = f.y[i] = f.dn[i] = f.dx[i] = 0.f;
                f.gate[i] = Sigmoid{1.f, 0.f};
            }
            if (!in) return;
            if (block) now.y[g].get(p.y.scales, k, f.y);
            if (gated) {
                float z[4];
                now.gate[g].get(p.gate.scales, k, z);
#pragma unroll
                for (int i = 0; i < 4; ++i) f.gate[i] = sigmoid2(z[i]);
            }
            if (pre) {
                now.x[g].get(p.x.scales, k, f.x);
                now.dn[g].get(false, k, f.dn);
            }
            if (p.d_x) now.dx[g].get(false, k, f.dx);
        };
        float s[6] = {};                                   // y^2, x^2, w_pre dn x, A dx, A w_pre dn, A x
        Floats f;
        f32x4 wpost, wres, wpre;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            weight(j, wpost, wres, wpre);
            floats(j, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float d = wpre[i] * f.dn[i], A = wpost[i] * wres[i] * (f.y[i] * f.gate[i].s);
                s[0] += f.y[i] * f.y[i];
                s[1] += f.x[i] * f.x[i];
                s[2] += d * f.x[i];
                s[3] += A * f.dx[i];
                s[4] += A * d;
                s[5] += A * f.x[i];
            }
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
        total(s);
        const float ry = p.post ? rstd_of(s[0] * inv_d + p.eps) : 1.f;
        const float rx = pre ? rstd_of(s[1] * inv_d + p.eps) : 0.f;
        const float mx = s[2] * rx * inv_d;                // mean of w_pre dn x^
        const float my = p.post ? (s[3] + rx * (s[4] - rx * mx * s[5])) * ry * inv_d : 0.f;
        if (!KEEP)
#pragma unroll
            for (int g = 0; g < NV; ++g) {
                now.x[g].hold();
                now.y[g].hold();
                now.gate[g].hold();
                now.dx[g].hold();
                now.dn[g].hold();
            }
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const unsigned c = channel(j);
            const int n = in ? max(0, min(4, p.D - (int)c)) : 0;
            if (!KEEP) {
                weight(j, wpost, wres, wpre);
                floats(j, f);
            }
            float G[4], dy[4], dgate[4];
            f32x4 sum = a_pre.get(j), post = a_post.get(j), res = a_res.get(j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float xh = f.x[i] * rx, yh = f.y[i] * ry, u = wpost[i] * yh;
                sum[i] += f.dn[i] * xh;
                G[i] = f.dx[i] + rx * (wpre[i] * f.dn[i] - xh * mx);
                const float dr = G[i] * wres[i], du = dr * f.gate[i].s;
                res[i] += G[i] * (f.gate[i].s * u);        // (times scale at the end)
                post[i] += du * yh;
                dgate[i] = dr * u * (f.gate[i].s * f.gate[i].r);
                dy[i] = ry * (wpost[i] * du - yh * my);
            }
            a_pre.put(j, sum);
            a_post.put(j, post);
            a_res.put(j, res);
            const auto store = [&](int m) {
                Raw4<X>::store(at_byte((X *)p.dx + r * p.D, c * sizeof(X)), m, G);
                if (block) Raw4<T>::store(at_byte((T *)p.dy + r * p.dy_stride, c * sizeof(T)), m, dy);
                if (gated) Raw4<T>::store(at_byte((T *)p.dgate + r * p.dgate_stride, c * sizeof(T)), m, dgate);
            };
            if (n > 0) {
                if (whole) store(4); else store(n);
            }
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) a_res.put(j, a_res.get(j) * p.scale);
    if (ROWS > 1) {                                        // the sides' sums, in their order (NQ 1)
        f32x4 *at = reinterpret_cast<f32x4 *>(s_mem) + t;
        if (side > 0) {
            at[(side - 1) * 3 * NT] = a_post.get(0);
            at[((side - 1) * 3 + 1) * NT] = a_res.get(0);
            at[((side - 1) * 3 + 2) * NT] = a_pre.get(0);
        }
        __syncthreads();
        if (side > 0) return;
        for (int k = 0; k < ROWS - 1; ++k) {
            a_post.put(0, a_post.get(0) + at[k * 3 * NT]);
            a_res.put(0, a_res.get(0) + at[(k * 3 + 1) * NT]);
            a_pre.put(0, a_pre.get(0) + at[(k * 3 + 2) * NT]);
        }
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const unsigned c = channel(j);
        const int n = max(0, min(4, p.D - (int)c));
        if (n == 0) continue;
        float *at = p.part + (size_t)blockIdx.x * p.D + c;
        const size_t other = (size_t)p.parts * p.D;
        const auto put = [&](f32x4 q, float *to) {
            const float v[4] = {q[0], q[1], q[2], q[3]};
            Raw4<float>::store(to, n, v);
        };
        if (p.dpost) put(a_post.get(j), at);
        if (p.dres) put(a_res.get(j), at + other);
        if (p.dpre) put(a_pre.get(j), at + 2 * other);
    }
}

// The weights' gradients from the workgroups' sums, in their order.  16 columns a workgroup (64 bytes of a row), 16 threads down
// each, eight rows on their way: with 64 columns and 4 threads, one row at a time, it took 36 us of 512 x 3 x 4096 sums.
__global__ __launch_bounds__(256) void norm_sum_kernel(const NormParams p)
{
    __shared__ double s_part[16][16];
    float *out = blockIdx.y == 0 ? p.dpost : blockIdx.y == 1 ? p.dres : p.dpre;
    if (!out) return;
    const double sum = column_sum(p.part + (size_t)blockIdx.y * p.parts * p.D, p.parts, p.D, s_part);
    const int c = blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x < 16 && c < p.D) out[c] = (float)sum;
}

template <typename T, typename X, int NW, int ROWS, int NCH> static hipError_t launch_fwd_t(const NormParams &p, hipStream_t stream)
{
    const int grid = (p.R + ROWS - 1) / ROWS, most = 256 * 16 / (NW * ROWS);         // 16 waves on each of 256 units
    hipLaunchKernelGGL((norm_fwd_kernel<T, X, NW, ROWS, NCH>), dim3(grid < most ? grid : most), dim3(64 * NW * ROWS), 0, stream, p);
    return hipGetLastError();
}

template <typename T, typename X, int NW, int ROWS, int NQ> static hipError_t launch_bwd_t(const NormParams &p, hipStream_t stream)
{
    static_assert(NW * ROWS == norm_waves(256 * NW * NQ) && ROWS == norm_rows(256 * NW * NQ), "as planned");
    constexpr size_t row = sizeof(float) * 256 * NW * NQ;                            // of floats
    constexpr size_t lds = row * (NQ == 1 ? 3 * (ROWS - 1) : NQ == 2 ? 3 : 2);
    if (p.R > 0) {
        if (lds > 0) {
            const hipError_t e = hipFuncSetAttribute((const void *)norm_bwd_kernel<T, X, NW, ROWS, NQ>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((norm_bwd_kernel<T, X, NW, ROWS, NQ>), dim3(p.parts), dim3(64 * NW * ROWS), lds, stream, p);
    }
    if (p.dpost || p.dres || p.dpre)
        hipLaunchKernelGGL(norm_sum_kernel, dim3((p.D + 15) / 16, 3), dim3(256), 0, stream, p);
    return hipGetLastError();
}

// Forward: 8 channels a lane, up to 16 waves a row, then twice that.
template <typename T, typename X> static hipError_t launch_fwd_x(const NormParams &p, hipStream_t stream)
{
    if (p.D <= 512) return launch_fwd_t<T, X, 1, 4, 1>(p, stream);
    if (p.D <= 1024) return launch_fwd_t<T, X, 2, 2, 1>(p, stream);
    if (p.D <= 2048) return launch_fwd_t<T, X, 4, 1, 1>(p, stream);
    if (p.D <= 4096) return launch_fwd_t<T, X, 8, 1, 1>(p, stream);
    if (p.D <= 8192) return launch_fwd_t<T, X, 16, 1, 1>(p, stream);
    return launch_fwd_t<T, X, 16, 1, 2>(p, stream);
}

// Backward: 4 channels a lane, up to 16 waves a row, then more.
template <typename T, typename X> static hipError_t launch_bwd_x(const NormParams &p, hipStream_t stream)
{
    if (p.D <= 256) return launch_bwd_t<T, X, 1, 4, 1>(p, stream);
    if (p.D <= 512) return launch_bwd_t<T, X, 2, 2, 1>(p, stream);
    if (p.D <= 1024) return launch_bwd_t<T, X, 4, 1, 1>(p, stream);
    if (p.D <= 2048) return launch_bwd_t<T, X, 8, 1, 1>(p, stream);
    if (p.D <= 4096) return launch_bwd_t<T, X, 16, 1, 1>(p, stream);
    if (p.D <= 8192) return launch_bwd_t<T, X, 16, 1, 2>(p, stream);
    return launch_bwd_t<T, X, 16, 1, 4>(p, stream);
}

hipError_t launch_norm_fwd(int is_bf16, int x_bf16, const NormParams &p, hipStream_t stream)
{
    if (!is_bf16) return launch_fwd_x<float, float>(p, stream);
    return x_bf16 ? launch_fwd_x<bf16, bf16>(p, stream) : launch_fwd_x<bf16, float>(p, stream);
}

hipError_t launch_norm_bwd(int is_bf16, int x_bf16, const NormParams &p, hipStream_t stream)
{
    if (!is_bf16) return launch_bwd_x<float, float>(p, stream);
    return x_bf16 ? launch_bwd_x<bf16, bf16>(p, stream) : launch_bwd_x<bf16, float>(p, stream);
}

}  // namespace kda
